/*
 * rope_partial.h -- C ABI of the MI355X (gfx950) in-place partial rotary
 * position embedding library, librope_partial.so.
 *
 * The operation ("CANN ops-transformer 算子详解：inplace_partial_rotary_mul
 * 原地部分旋转位置编码", sections 功能与计算公式 and 约束说明; rotate_half
 * pairing from "ANE实战RoPE位置编码在MIL中的纯ANE实现", section 先搞懂RoPE):
 *
 *   x has shape (B,S,N,D), row-major and contiguous (BSND). Only the lanes
 *   [start,end) of the last dimension are rotated, in place; every other lane
 *   keeps its bytes. With L = end - start and slice lane j in [0,L):
 *     interleave  (mode 1): partner p(j) = j xor 1,   sign s(j) = -1 if j even
 *     rotate_half (mode 0): partner p(j) = j +- L/2,  sign s(j) = -1 if j < L/2
 *     rotary coefficient (mode c >= 2, even, dividing L; "ascend-transformer-
 *     boost 的 MlaPreprocessOperation", section 2, qRotaryCoeff/kRotaryCoeff:
 *     2 is the half rotation, 4 or headDim also allowed): the slice in c
 *     parts of H = L/c lanes, lane k of part 2g paired with lane k of part
 *     2g+1: p(j) = j +- H, s(j) = -1 in an even part. c = 2 is rotate_half,
 *     c = L interleave.
 *   forward : y_j  = x_j * r1_j + s(j) * x_p(j) * r2_j
 *   backward: dx_j = g_j * r1_j - s(j) * g_p(j) * r2_p(j)
 *   (the backward is the transposed Jacobian of the forward -- the gradient
 *   with respect to x, section 自动微分说明 -- which equals rotating by -θ
 *   when the tables hold one angle per pair.)
 *   r1 (cos) and r2 (sin) are read at the broadcast index of (b,s,n,j).
 *   Arithmetic is fp32 (the page's mixed-precision paragraph: inputs are
 *   cast to fp32 for the multiply-add and written back with round-to-
 *   nearest-even). For 16-bit x each product is rounded to fp32, the sum is
 *   rounded to fp32, and the result is rounded to nearest-even to the
 *   storage type; with 16-bit tables the products are exact, so that is one
 *   rounding of the exact sum. For fp32 x the multiply-add may be fused.
 *
 * Memory: every pointer is a device pointer on the current HIP device. The
 * caller owns all memory; the library allocates nothing and keeps no state
 * but a per-device cache of the compute-unit count. Calls are asynchronous on
 * `stream` (a hipStream_t; NULL is the null stream). A call that returns an
 * error before the launch has not touched device memory.
 */
#ifndef ROPE_PARTIAL_H
#define ROPE_PARTIAL_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* symbols of the C ABI; everything else in the library is hidden */
#define ROPE_API __attribute__((visibility("default")))

/*
 * Status codes. The classes follow the aclnn convention described on the
 * CANN ops-transformer page on aclnnMoeTokenUnpermuteWithEpGrad, section
 * 六、返回值与错误码 (a NULL required tensor, a parameter outside the supported
 * range, an inner error); the numbers are this library's own.
 */
typedef enum rope_status {
    ROPE_OK = 0,
    ROPE_ERR_NULLPTR = 1,      /* a required pointer is NULL                   */
    ROPE_ERR_INVALID = 2,      /* an argument breaks the constraints below     */
    ROPE_ERR_UNSUPPORTED = 3,  /* a valid combination the library does not run */
    ROPE_ERR_RUNTIME = 4       /* the HIP runtime reported an error            */
} rope_status_t;

typedef enum rope_dtype {
    ROPE_DTYPE_F32 = 0,
    ROPE_DTYPE_F16 = 1,
    ROPE_DTYPE_BF16 = 2
} rope_dtype_t;

/* rotary modes; interleave keeps the integer the CANN interface gives it.
 * A mode value c >= 2 is a rotary coefficient (above). */
#define ROPE_MODE_ROTATE_HALF 0
#define ROPE_MODE_INTERLEAVE 1

/* largest supported head dimension D (the page's D limit) */
#define ROPE_D_LIMIT 1024

/* ======================== cos/sin from tables ======================== */

/*
 * rope_partial_fwd_inplace -- rotate x[..., start:end) in place (forward).
 *
 *   x            device buffer of B*S*N*D elements of `dtype`, contiguous
 *                BSND; 16-byte alignment enables the vector kernels.
 *   x_shape      host array {B, S, N, D}; each >= 0, D even, D <= 1024.
 *   dtype        storage type of x.
 *   r1, r2       device buffers: cos and sin tables of `table_dtype`.
 *   r*_shape     host arrays, 4-D; r*_shape[3] == L and, for k < 3,
 *                r*_shape[k] is 1 (broadcast) or x_shape[k]. This admits the
 *                layouts the page lists (BSND, B1ND, B11D, 111D, BS1D) and
 *                any other broadcast of the same rule.
 *   r*_strides   host arrays, strides in elements, each >= 0;
 *                r*_strides[3] must be 1. The stride of a size-1 dimension
 *                is ignored (this is what torch's expand() produces).
 *   table_dtype  storage type of r1 and r2 (any of the three, independent
 *                of dtype; the page's mixed case is 16-bit x with fp32
 *                tables).
 *   mode         ROPE_MODE_INTERLEAVE, ROPE_MODE_ROTATE_HALF, or a rotary
 *                coefficient c: even, >= 2, dividing L (when L > 0).
 *   partial_slice host array {start, end} or NULL, which means {0, 0}:
 *                0 <= start <= end <= D and L = end - start even.
 *   stream       hipStream_t to launch on, or NULL.
 *
 * Checks, in this order: scalar arguments (ROPE_ERR_NULLPTR for a NULL
 * x_shape, ROPE_ERR_INVALID otherwise); then an empty tensor (B*S*N*D == 0)
 * or an empty slice (L == 0) returns ROPE_OK at once without reading any
 * pointer (no-op, as the page specifies for forward and backward); then NULL
 * data or table pointers (ROPE_ERR_NULLPTR); then table shapes and strides
 * (ROPE_ERR_INVALID); finally the launch (ROPE_ERR_RUNTIME if HIP reports
 * an error). ROPE_ERR_UNSUPPORTED is not returned by this call (only
 * rope_proj_fwd returns it, for shapes its kernel does not tile).
 * Overlapping x with r1 or r2 is undefined. Results are deterministic: each
 * element is computed by one thread from the same inputs on every call.
 */
ROPE_API rope_status_t rope_partial_fwd_inplace(
    void* x, const int64_t x_shape[4], rope_dtype_t dtype,
    const void* r1, const int64_t r1_shape[4], const int64_t r1_strides[4],
    const void* r2, const int64_t r2_shape[4], const int64_t r2_strides[4],
    rope_dtype_t table_dtype, int64_t mode, const int64_t partial_slice[2],
    void* stream);

/*
 * rope_partial_bwd_inplace -- the backward of rope_partial_fwd_inplace:
 * x holds the incoming gradient dy on entry and dx on return (in place).
 * Arguments, checks and no-op rules are those of the forward; r1 and r2
 * receive no gradient (the page's autograd returns None for them).
 */
ROPE_API rope_status_t rope_partial_bwd_inplace(
    void* x, const int64_t x_shape[4], rope_dtype_t dtype,
    const void* r1, const int64_t r1_shape[4], const int64_t r1_strides[4],
    const void* r2, const int64_t r2_shape[4], const int64_t r2_strides[4],
    rope_dtype_t table_dtype, int64_t mode, const int64_t partial_slice[2],
    void* stream);

/*
 * rope_partial_fwd_out / rope_partial_bwd_out -- the same operation out of
 * place: y (dx) receives x (dy) with the lanes [start,end) rotated, forward
 * or backward as above, and every other lane copied bit for bit; x is not
 * modified. The page's autograd backward (section 自动微分说明) needs this
 * form: the incoming gradient may be shared with other consumers, so it
 * cannot be rotated in place, and one pass that reads it and writes the
 * result moves less memory than a copy followed by the in-place call.
 *
 *   y            device buffer for the result: B*S*N*D elements of `dtype`,
 *                contiguous BSND, owned by the caller. y == x is the
 *                in-place call; any other overlap of y and x is an error.
 *   x            device buffer of the input, same shape and type.
 *   Other arguments are those of rope_partial_fwd_inplace.
 *
 * Checks, in this order: the scalar arguments (as above); an empty tensor
 * returns ROPE_OK without reading any pointer; NULL y or x
 * (ROPE_ERR_NULLPTR); y and x overlapping without being equal
 * (ROPE_ERR_INVALID); an empty slice (L == 0) then copies x to y without
 * looking at the tables, which may be NULL; otherwise the table pointers
 * and geometry are checked as above. When both buffers are 16-byte aligned
 * (and the vector kernel's size limits hold) one kernel reads x and writes
 * y; otherwise x is copied to y on `stream` and y is rotated in place.
 */
ROPE_API rope_status_t rope_partial_fwd_out(
    void* y, const void* x, const int64_t x_shape[4], rope_dtype_t dtype,
    const void* r1, const int64_t r1_shape[4], const int64_t r1_strides[4],
    const void* r2, const int64_t r2_shape[4], const int64_t r2_strides[4],
    rope_dtype_t table_dtype, int64_t mode, const int64_t partial_slice[2],
    void* stream);

ROPE_API rope_status_t rope_partial_bwd_out(
    void* dx, const void* dy, const int64_t x_shape[4], rope_dtype_t dtype,
    const void* r1, const int64_t r1_shape[4], const int64_t r1_strides[4],
    const void* r2, const int64_t r2_shape[4], const int64_t r2_strides[4],
    rope_dtype_t table_dtype, int64_t mode, const int64_t partial_slice[2],
    void* stream);

/* largest tensor count of the _multi entry points */
#define ROPE_MULTI_MAX 4

/*
 * rope_partial_fwd_inplace_multi / rope_partial_bwd_inplace_multi -- rotate
 * `count` tensors that share one pair of tables (for example the Q and K of
 * one attention layer, whose head counts differ under grouped-query
 * attention) with one call; the result is that of calling the single-tensor
 * entry point on xs[0], xs[1], ... in order on `stream`. When every tensor
 * takes the same vector kernel, all of them run in a single kernel launch
 * (one launch overhead, tables shared in cache). "ANE实战RoPE位置编码在MIL中的
 * 纯ANE实现", section 第二步, applies the same rotation to Q and to K.
 *
 *   count      0..ROPE_MULTI_MAX; 0 is a no-op.
 *   xs         host array of `count` device pointers.
 *   x_shapes   host array of `count` shapes {B, S, N, D}.
 *   Other arguments are those of rope_partial_fwd_inplace and apply to every
 *   tensor: the tables must broadcast against each tensor's slice.
 *
 * Every tensor is checked before anything is launched: on an error no
 * memory has been touched, and rope_last_error() names the tensor.
 * count outside [0, ROPE_MULTI_MAX] is ROPE_ERR_INVALID; NULL xs or x_shapes
 * with count > 0 is ROPE_ERR_NULLPTR. Tensors that share any byte (the same
 * tensor passed twice included) are ROPE_ERR_INVALID, checked after every
 * tensor's own checks and before any launch: one fused launch would read
 * and write the shared bytes from two threads at once.
 */
ROPE_API rope_status_t rope_partial_fwd_inplace_multi(
    int32_t count, void* const xs[], const int64_t x_shapes[][4], rope_dtype_t dtype,
    const void* r1, const int64_t r1_shape[4], const int64_t r1_strides[4],
    const void* r2, const int64_t r2_shape[4], const int64_t r2_strides[4],
    rope_dtype_t table_dtype, int64_t mode, const int64_t partial_slice[2],
    void* stream);

ROPE_API rope_status_t rope_partial_bwd_inplace_multi(
    int32_t count, void* const xs[], const int64_t x_shapes[][4], rope_dtype_t dtype,
    const void* r1, const int64_t r1_shape[4], const int64_t r1_strides[4],
    const void* r2, const int64_t r2_shape[4], const int64_t r2_strides[4],
    rope_dtype_t table_dtype, int64_t mode, const int64_t partial_slice[2],
    void* stream);

/* ====================== cos/sin from positions ====================== */

/*
 * rope_partial_fwd_inplace_pos / rope_partial_bwd_inplace_pos -- the same
 * in-place operation with cos and sin computed from positions instead of
 * read from tables. "ANE实战RoPE位置编码在MIL中的纯ANE实现", section 第一步,
 * builds the tables from θ = p / base^(2i/h) for position p and pair i;
 * here, for the row (b,s,n) and the slice's pair i:
 *   θ = (double)positions[b, s] * inv_freq[i]      (one double product)
 *   c = RN_T(cos θ),  s = RN_T(sin θ)             (double precision, then
 *                                                   one rounding to nearest
 *                                                   even to table_dtype T)
 * placed as a table would hold them (interleave: lanes 2i and 2i+1;
 * rotate_half: lanes i and i + L/2). The result is that of the table entry
 * points given tables (Bp, S, 1, L) of type T with these values, up to the
 * last-bit differences of two double-precision cos/sin implementations,
 * which change a rounding to T only for values within about 2^-52 of a
 * midpoint of T.
 *
 *   positions          device int64 array; the position of (b,s) is
 *                      positions[b*positions_strides[0] + s*positions_strides[1]].
 *   positions_shape    host {Bp, S}: Bp is 1 (one row of positions for every
 *                      batch) or B, and S is x's S.
 *   positions_strides  host, in elements, each >= 0; a size-1 dimension's
 *                      stride is ignored.
 *   inv_freq           device array of L/2 doubles, pair i's frequency
 *                      (base^(-2i/L) for the page's recipe; any values, e.g.
 *                      scaled frequencies, are taken as given).
 *   table_dtype        T, the type cos and sin are rounded to (any of the
 *                      three, independent of dtype).
 *   Other arguments are those of rope_partial_fwd_inplace.
 *
 * Checks, in this order: the scalar arguments; an empty tensor or slice
 * returns ROPE_OK at once; NULL x, positions, inv_freq, positions_shape or
 * positions_strides (ROPE_ERR_NULLPTR); positions_shape not {1 or B, S}, a
 * negative stride, or offsets beyond 64 bits (ROPE_ERR_INVALID). Memory as
 * for the table entry points: asynchronous on `stream`, nothing allocated.
 */
ROPE_API rope_status_t rope_partial_fwd_inplace_pos(
    void* x, const int64_t x_shape[4], rope_dtype_t dtype,
    const int64_t* positions, const int64_t positions_shape[2], const int64_t positions_strides[2],
    const double* inv_freq, rope_dtype_t table_dtype, int64_t mode, const int64_t partial_slice[2],
    void* stream);

ROPE_API rope_status_t rope_partial_bwd_inplace_pos(
    void* x, const int64_t x_shape[4], rope_dtype_t dtype,
    const int64_t* positions, const int64_t positions_shape[2], const int64_t positions_strides[2],
    const double* inv_freq, rope_dtype_t table_dtype, int64_t mode, const int64_t partial_slice[2],
    void* stream);

/*
 * rope_partial_fwd_out_pos / rope_partial_bwd_out_pos -- the position forms
 * out of place: y receives x with its slice rotated, cos and sin computed
 * from positions exactly as rope_partial_fwd_inplace_pos does, and x is left
 * unchanged. y == x is the in-place call. An empty slice copies x to y.
 *
 *   y, x         device buffers of B*S*N*D elements of `dtype`, contiguous
 *                BSND; y is written, x is read. With both 16-byte aligned
 *                one kernel reads x and writes y in one pass; otherwise x is
 *                copied to y and y is rotated in place.
 *   Other arguments are those of rope_partial_fwd_inplace_pos.
 *
 * Checks, in this order: the scalar arguments; an empty tensor returns
 * ROPE_OK at once; NULL y or x (ROPE_ERR_NULLPTR); y and x overlapping
 * without being the same buffer (ROPE_ERR_INVALID); an empty slice copies;
 * then the checks of positions, positions_shape, positions_strides and
 * inv_freq of the in-place form. Asynchronous on `stream`; nothing is
 * allocated.
 */
ROPE_API rope_status_t rope_partial_fwd_out_pos(
    void* y, const void* x, const int64_t x_shape[4], rope_dtype_t dtype,
    const int64_t* positions, const int64_t positions_shape[2], const int64_t positions_strides[2],
    const double* inv_freq, rope_dtype_t table_dtype, int64_t mode, const int64_t partial_slice[2],
    void* stream);

ROPE_API rope_status_t rope_partial_bwd_out_pos(
    void* y, const void* x, const int64_t x_shape[4], rope_dtype_t dtype,
    const int64_t* positions, const int64_t positions_shape[2], const int64_t positions_strides[2],
    const double* inv_freq, rope_dtype_t table_dtype, int64_t mode, const int64_t partial_slice[2],
    void* stream);

/*
 * rope_partial_fwd_inplace_pos_multi / rope_partial_bwd_inplace_pos_multi
 * -- the position forms for `count` tensors that share one set of positions
 * (the Q and K of one attention layer, whose head counts may differ); the
 * result is that of calling rope_partial_fwd_inplace_pos on xs[0], xs[1],
 * ... in order on `stream`. When the tensors share B, S and D and take the
 * vector kernel, all of them run in a single launch that evaluates each
 * pair's cos and sin once per position for every tensor. "ANE实战RoPE位置编码
 * 在MIL中的纯ANE实现", section 第二步, applies the same rotation to Q and K.
 *
 *   count      0..ROPE_MULTI_MAX; 0 is a no-op.
 *   xs         host array of `count` device pointers.
 *   x_shapes   host array of `count` shapes {B, S, N, D}.
 *   Other arguments are those of rope_partial_fwd_inplace_pos and apply to
 *   every tensor: positions_shape must fit each tensor's B and S.
 *
 * Every tensor is checked before anything is launched: on an error no
 * memory has been touched, and rope_last_error() names the tensor. count
 * outside [0, ROPE_MULTI_MAX] is ROPE_ERR_INVALID; NULL xs or x_shapes with
 * count > 0 is ROPE_ERR_NULLPTR. Tensors that share any byte are
 * ROPE_ERR_INVALID, as for rope_partial_fwd_inplace_multi.
 */
ROPE_API rope_status_t rope_partial_fwd_inplace_pos_multi(
    int32_t count, void* const xs[], const int64_t x_shapes[][4], rope_dtype_t dtype,
    const int64_t* positions, const int64_t positions_shape[2], const int64_t positions_strides[2],
    const double* inv_freq, rope_dtype_t table_dtype, int64_t mode, const int64_t partial_slice[2],
    void* stream);

ROPE_API rope_status_t rope_partial_bwd_inplace_pos_multi(
    int32_t count, void* const xs[], const int64_t x_shapes[][4], rope_dtype_t dtype,
    const int64_t* positions, const int64_t positions_shape[2], const int64_t positions_strides[2],
    const double* inv_freq, rope_dtype_t table_dtype, int64_t mode, const int64_t partial_slice[2],
    void* stream);

/* ================= cos/sin from positions on several axes ================= */

/* most axes of one call */
#define ROPE_AXES_MAX 4

/*
 * rope_partial_{fwd,bwd}_inplace_axes, _out_axes, _inplace_axes_multi -- the
 * position forms with positions on several axes (time, height and width of
 * images and video): pair i of the slice belongs to the axis pair_axes[i]
 * and turns by
 *   θ = (double)positions[pair_axes[i], b, s] * inv_freq[i]
 * cos and sin as for rope_partial_fwd_inplace_pos. Which pairs an axis takes
 * (blocks, dealt in turn, any other order) and whether the frequencies run
 * over all pairs or over each axis's own is the caller's choice of pair_axes
 * and inv_freq.
 *
 *   positions          device int64 array; the position of (b,s) on axis k is
 *                      positions[k*positions_strides[0] +
 *                      b*positions_strides[1] + s*positions_strides[2]].
 *   positions_shape    host {A, Bp, S}: A axes, 1 to ROPE_AXES_MAX; Bp is 1
 *                      (every batch alike) or B, and S is x's S.
 *   positions_strides  host, in elements, each >= 0; a size-1 dimension's
 *                      stride is ignored.
 *   pair_axes          host array of L/2 axes, each in [0, A), read during
 *                      the call.
 *   Other arguments, overlap rules, no-ops and memory are those of the _pos
 *   entry point of the same form.
 *
 * Checks: those of the _pos entry points in their order; pair_axes NULL
 * (ROPE_ERR_NULLPTR) after the other pointers; A outside [1, ROPE_AXES_MAX]
 * before the other dimensions, and a pair's axis outside [0, A) last
 * (ROPE_ERR_INVALID).
 */
ROPE_API rope_status_t rope_partial_fwd_inplace_axes(
    void* x, const int64_t x_shape[4], rope_dtype_t dtype, const int64_t* positions,
    const int64_t positions_shape[3], const int64_t positions_strides[3], const double* inv_freq,
    const int32_t* pair_axes, rope_dtype_t table_dtype, int64_t mode, const int64_t partial_slice[2],
    void* stream);

ROPE_API rope_status_t rope_partial_bwd_inplace_axes(
    void* x, const int64_t x_shape[4], rope_dtype_t dtype, const int64_t* positions,
    const int64_t positions_shape[3], const int64_t positions_strides[3], const double* inv_freq,
    const int32_t* pair_axes, rope_dtype_t table_dtype, int64_t mode, const int64_t partial_slice[2],
    void* stream);

ROPE_API rope_status_t rope_partial_fwd_out_axes(
    void* y, const void* x, const int64_t x_shape[4], rope_dtype_t dtype, const int64_t* positions,
    const int64_t positions_shape[3], const int64_t positions_strides[3], const double* inv_freq,
    const int32_t* pair_axes, rope_dtype_t table_dtype, int64_t mode, const int64_t partial_slice[2],
    void* stream);

ROPE_API rope_status_t rope_partial_bwd_out_axes(
    void* y, const void* x, const int64_t x_shape[4], rope_dtype_t dtype, const int64_t* positions,
    const int64_t positions_shape[3], const int64_t positions_strides[3], const double* inv_freq,
    const int32_t* pair_axes, rope_dtype_t table_dtype, int64_t mode, const int64_t partial_slice[2],
    void* stream);

ROPE_API rope_status_t rope_partial_fwd_inplace_axes_multi(
    int32_t count, void* const xs[], const int64_t x_shapes[][4], rope_dtype_t dtype, const int64_t* positions,
    const int64_t positions_shape[3], const int64_t positions_strides[3], const double* inv_freq,
    const int32_t* pair_axes, rope_dtype_t table_dtype, int64_t mode, const int64_t partial_slice[2],
    void* stream);

ROPE_API rope_status_t rope_partial_bwd_inplace_axes_multi(
    int32_t count, void* const xs[], const int64_t x_shapes[][4], rope_dtype_t dtype, const int64_t* positions,
    const int64_t positions_shape[3], const int64_t positions_strides[3], const double* inv_freq,
    const int32_t* pair_axes, rope_dtype_t table_dtype, int64_t mode, const int64_t partial_slice[2],
    void* stream);

/* ===================== paged key/value cache, quantised ===================== */

/* how a cache holds its lanes */
typedef enum rope_cache_format {
    ROPE_CACHE_F32 = 0,   /* the storage types, as rope_dtype_t: no scales */
    ROPE_CACHE_F16 = 1,
    ROPE_CACHE_BF16 = 2,
    ROPE_CACHE_E4M3 = 3,  /* 8-bit float, 4 exponent and 3 fraction bits, largest value 448 */
    ROPE_CACHE_INT8 = 4,  /* -127 to 127 */
    ROPE_CACHE_INT4 = 5   /* -7 to 7, two's complement; lane 2i in the low half of byte i, 2i+1 in the high half */
} rope_cache_format_t;

/*
 * A paged cache of keys or values: `pages` pages of `page_size` slots, each
 * slot holding `heads` rows of `dim` lanes. Slot number t is slot t %
 * page_size of page t / page_size. A quantised format keeps one fp32 scale
 * for every `group` lanes of a row: lane j stands for code[j] * scale[j / group].
 */
typedef struct rope_cache {
    void* data;               /* device; the lanes of a row are consecutive */
    float* scales;            /* device; the scales of a row are consecutive; NULL for the storage types */
    int32_t format;           /* rope_cache_format_t */
    int64_t pages, page_size, heads, dim;
    int64_t group;            /* lanes per scale: even, divides dim (ignored for the storage types) */
    int64_t strides[3];       /* BYTES from one page, slot and head to the next */
    int64_t scale_strides[3]; /* floats from one page, slot and head to the next */
} rope_cache_t;

/* Rows of a (B, S, N, D) tensor whose last dimension is consecutive. */
typedef struct rope_rows {
    void* data;               /* device */
    int64_t N, D;
    int64_t strides[3];       /* elements from one b, s and n to the next, each >= 0 */
} rope_rows_t;

/*
 * rope_cache_write -- rotate the keys of B x S tokens and write them, with
 * the values, to their slots of a cache, quantised; and rotate the queries
 * beside them. One launch. For each token (b,s) with slot t = slots[b,s] in
 * [0, pages * page_size):
 *   z = k[b,s,h,:] with its slice rotated from positions (forward, fp32, as
 *       rope_partial_fwd_inplace_axes; never rounded to the storage type)
 *       when rotate_k is not 0, else k itself;
 *   quantised formats, for each group of lanes: m = the largest |z_j| of the
 *       finite lanes, scale = m / Q rounded to fp32 and at least 2^-100 (1
 *       when m = 0), code_j = z_j / scale (the exact quotient of the two
 *       numbers) rounded once to the nearest code, ties to even. Q is 448
 *       (e4m3), 127 or 7. An infinite lane takes the code of +-m, a NaN lane
 *       NaN (e4m3) or 0: it does not touch the lanes beside it;
 *   storage types: z rounded once.
 * v is written the same way without rotation. Every other slot keeps its
 * bytes: a token whose slot is negative or past the cache is not written
 * (the padding of a batch). Slots of one call must differ; what a slot given
 * twice holds afterwards is unspecified. q is rotated in place, for every
 * token.
 *
 *   B, S        tokens; dtype: storage type of q, k and v.
 *   q, v        NULL when there is none. q has k's D.
 *   k, v        (B, S, heads, dim) of their cache; read only; any strides.
 *   v_cache     NULL exactly when v is; pages and page_size of k_cache.
 *               k and v caches: formats that are quantised, or `dtype`.
 *   slots       device int64, at b*slots_strides[0] + s*slots_strides[1].
 *   positions, positions_shape {A, Bp, S}, positions_strides, inv_freq,
 *   pair_axes, table_dtype, mode, partial_slice
 *               as for rope_partial_fwd_inplace_axes; pair_axes may be NULL
 *               when A is 1. With an empty slice, or neither q nor rotate_k,
 *               nothing is rotated and positions are not looked at.
 *
 * q must not share a byte with itself (rows that overlap are refused), nor
 * with k, v or the caches, nor k and v with the caches (not checked: the rows
 * of one fused projection lie between each other). Checks, in order: B, S, dtype, k, k_cache, v and
 * v_cache present (ROPE_ERR_NULLPTR); mode, slice and types as
 * rope_partial_fwd_inplace on k's shape; the caches' fields; q and v against
 * them; strides; no token or no lanes: ROPE_OK; NULL data; then positions.
 * ROPE_ERR_UNSUPPORTED: 2^31 rows of q, k and v or more. Asynchronous on
 * `stream`; nothing is allocated; deterministic.
 */
ROPE_API rope_status_t rope_cache_write(
    int64_t B, int64_t S, rope_dtype_t dtype, const rope_rows_t* q, const rope_rows_t* k, const rope_rows_t* v,
    const rope_cache_t* k_cache, const rope_cache_t* v_cache, const int64_t* slots, const int64_t slots_strides[2],
    const int64_t* positions, const int64_t positions_shape[3], const int64_t positions_strides[3],
    const double* inv_freq, const int32_t* pair_axes, rope_dtype_t table_dtype, int64_t mode,
    const int64_t partial_slice[2], int32_t rotate_k, void* stream);

/*
 * rope_cache_read -- read cached tokens back: for every sequence b and s in
 * [0, min(lengths[b], S)), token t = starts[b] + s of the sequence is slot
 * t % page_size of page block_table[b, t / page_size], and
 *   out[b,s,h,j] = code_j * scale (fp32), its slice rotated from positions
 *                  when they are given, rounded once to `dtype`.
 * Keys stored unrotated are rotated this way, and rotated ones moved to
 * other positions. Every other row of out keeps its bytes: s >= lengths[b],
 * tokens before 0 or past the block table, and pages outside [0, pages).
 *
 *   out           (B, S, heads, dim) rows of `dtype`; rows must not overlap
 *                 each other, nor any input (the latter is not checked).
 *   cache         any quantised format, or the format of `dtype`.
 *   block_table   device int32, B rows of table_pages pages, row b at
 *                 b * table_stride.
 *   lengths       device int32 (B); starts: device int32 (B) or NULL (0).
 *   positions     NULL: nothing is rotated and the arguments up to
 *                 partial_slice but table_dtype and mode are not looked at;
 *                 else as for rope_cache_write, for out's (b,s).
 *
 * Checks, in order: as rope_cache_write's for its arguments; an empty out is
 * ROPE_OK; NULL data, block_table or lengths; positions.
 */
ROPE_API rope_status_t rope_cache_read(
    int64_t B, int64_t S, rope_dtype_t dtype, const rope_rows_t* out, const rope_cache_t* cache,
    const int32_t* block_table, int64_t table_pages, int64_t table_stride, const int32_t* lengths,
    const int32_t* starts, const int64_t* positions, const int64_t positions_shape[3],
    const int64_t positions_strides[3], const double* inv_freq, const int32_t* pair_axes, rope_dtype_t table_dtype,
    int64_t mode, const int64_t partial_slice[2], void* stream);

/* most sequences of one rope_cache_reserve */
#define ROPE_RESERVE_MAX 16384

/*
 * rope_cache_reserve -- a step's bookkeeping of a paged cache, on the device:
 * pages are given to sequences that grow and taken back from those that
 * shrink or end, and the new tokens get their slots and positions (what
 * rope_cache_write and the position calls take). With pages(n) = ceil(n /
 * page_size):
 *   1. For every b with counts[b] < 0, in order: the sequence keeps k =
 *      max(0, lengths[b] + counts[b]) tokens. The pages of columns [pages(k),
 *      pages(lengths[b])) of its row go to the end of the free list, in order
 *      (what would pass its capacity is dropped), and -1 takes their place.
 *   2. For every b with 0 < counts[b] <= S whose lengths[b] + counts[b] tokens
 *      fit in its row of the table: it needs the columns [pages(lengths[b]),
 *      pages(lengths[b] + counts[b])). It gets them from the end of the free
 *      list, the first column the last page, if it needs none, or the pages
 *      needed by it and every sequence before it (served or not) are no more
 *      than the list holds. Otherwise, or where the row is too short, nothing
 *      of it changes.
 *   granted[b]     what is added to lengths[b]: counts[b] where it was served,
 *                  minus the tokens dropped in 1, else 0.
 *   positions[b,s] k + s in 1, else lengths[b] (before) + s; for every s < S.
 *   slots[b,s]     for s < granted[b] the slot of token positions[b,s]: its
 *                  page * page_size + its place in it; else, or where the page
 *                  is negative, -1.
 * A row whose length is negative or past its columns is left alone (granted
 * 0). Every other entry of the table, and the free list's places behind its
 * count, keep their values.
 *
 *   block_table   device int32, B rows of table_pages pages, row b at
 *                 b * table_stride >= table_pages; changed in place, as are
 *   lengths       device int32 (B),
 *   free_pages    device int32 (free_capacity): a list of free pages of
 *   free_count    device int32 (1) entries.
 *   counts        device int32 (B).
 *   slots, positions  device int64 (B, S), contiguous; granted: int32 (B).
 *
 * The arrays must not overlap. Checks: sizes (ROPE_ERR_INVALID; S at least 1;
 * B of 0 is ROPE_OK; more than ROPE_RESERVE_MAX sequences, or B * S, page_size,
 * free_capacity or table_pages of 2^31 or more: ROPE_ERR_UNSUPPORTED), NULL
 * pointers, alignment. Asynchronous on `stream`; nothing is allocated;
 * deterministic. Calls on the same table must follow each other.
 */
ROPE_API rope_status_t rope_cache_reserve(
    int64_t B, int64_t S, int32_t* block_table, int64_t table_pages, int64_t table_stride, int32_t* lengths,
    const int32_t* counts, int32_t* free_pages, int64_t free_capacity, int32_t* free_count, int64_t page_size,
    int64_t* slots, int64_t* positions, int32_t* granted, void* stream);

/*
 * rope_cache_attention -- attention of a step's new tokens over a paged cache
 * held in 4 bits. Sequence b has lengths[b] cached tokens, the last counts[b]
 * of which are the new ones whose queries are given: query s < counts[b]
 * stands at token lengths[b] - counts[b] + s. With k_t and v_t the cached rows
 * (code * scale) of the cached head that query head h belongs to (h / (q heads
 * / heads)):
 *   x_t = scale * q[b,s,h,:] . k_t
 *   out[b,s,h,:] = sum_t exp(x_t) v_t / sum_t exp(x_t)
 * over the tokens t in [0, lengths[b]) that the block table holds (row b's
 * page t / page_size, in [0, pages)) and, when causal is not 0, t no later than
 * the query's own. A row that sees no token is 0. Rows s >= counts[b] of out
 * keep their bytes.
 * Products with q are exact and summed in fp32, as are the softmax's sums
 * and its products with v; 16-bit outputs may round exp(x_t) times v's scale
 * to 11 bits before the product. out is rounded once. Long sequences are
 * summed in parts, whose size follows from the lengths of all. A scale that is
 * infinite or NaN reaches the rows that see its token, and no other.
 *
 *   B, S          tokens of q and out; dtype: their storage type.
 *   out, q        (B, S, heads of q, lanes of v or k) rows; out's must not
 *                 overlap each other or an input (the latter is not checked).
 *   k_cache, v_cache  ROPE_CACHE_INT4, the same pages, page_size and heads
 *                 (which divide q's); dim and group may differ.
 *   block_table, table_pages, table_stride   as for rope_cache_read.
 *   lengths       device int32 (B); counts: device int32 (B) or NULL (S).
 *                 Counts outside [0, S] are taken as the nearest of the two.
 *   scale         positive.
 *   workspace     device buffer of workspace_bytes, 16-byte aligned, used
 *                 during the call: at least rope_cache_attention_workspace(B,
 *                 S, heads of q, heads, lanes of v). Two calls that may run at
 *                 once need one each. Not looked at where that is 0.
 *
 * Checks, in order: q's dimensions and type; the caches' fields, formats
 * (ROPE_ERR_UNSUPPORTED unless ROPE_CACHE_INT4) and shapes; strides; scale; an
 * empty q is ROPE_OK; NULL or misaligned pointers; the workspace.
 * ROPE_ERR_UNSUPPORTED: 2^31 rows or more. Asynchronous on `stream`; nothing
 * is allocated; deterministic (the same call gives the same bits; a sequence in
 * another batch may differ in its last ones).
 */
ROPE_API rope_status_t rope_cache_attention(
    int64_t B, int64_t S, rope_dtype_t dtype, const rope_rows_t* out, const rope_rows_t* q, const rope_cache_t* k_cache,
    const rope_cache_t* v_cache, const int32_t* block_table, int64_t table_pages, int64_t table_stride,
    const int32_t* lengths, const int32_t* counts, double scale, int32_t causal, void* workspace,
    int64_t workspace_bytes, void* stream);

/* Bytes of workspace that a rope_cache_attention of this shape needs, however
 * many tokens are cached (0 when the arguments are out of range). */
ROPE_API int64_t rope_cache_attention_workspace(int64_t B, int64_t S, int64_t q_heads, int64_t heads, int64_t v_dim);

/* ============== norms of query and key heads with their rotation ============== */

/*
 * rope_qk_norm_fwd -- RMS norms of the heads of Q and K and their rotation in
 * one pass: for every row x of D lanes
 *     n_j = x_j / sqrt(mean(x^2) + eps) * weight_j
 *     out = n with its slice rotated from positions, forward, as
 *           rope_partial_fwd_inplace_axes rotates fp32 data
 * in fp32, rounded once to `dtype`. The mean is over all D lanes.
 *
 *   B, S, dtype   tokens; storage type of q, k and their results.
 *   q, k          (B, S, heads, D) rows, read; any strides (slices of a fused
 *                 projection's output). k and k_out are NULL when there is no
 *                 k. Heads may differ, D may not.
 *   q_out, k_out  rows of the same shapes; theirs must not overlap each other.
 *                 q_out may be q, with its strides, and k_out k (in place).
 *   q_weight, k_weight  device arrays of D weight_dtype numbers, or NULL: ones.
 *   eps           finite, not negative.
 *   positions, ... partial_slice  as for rope_cache_write; positions NULL, or
 *                 an empty slice: nothing is rotated.
 *
 * Checks, in order: NULL rows; q's dimensions, types, mode and slice; eps; the
 * other rows' shapes and strides; 2^31 rows or more (ROPE_ERR_UNSUPPORTED); no
 * row: ROPE_OK; NULL or misaligned data; positions. Asynchronous on `stream`;
 * nothing is allocated; deterministic.
 */
ROPE_API rope_status_t rope_qk_norm_fwd(
    int64_t B, int64_t S, rope_dtype_t dtype, const rope_rows_t* q_out, const rope_rows_t* k_out, const rope_rows_t* q,
    const rope_rows_t* k, const void* q_weight, const void* k_weight, rope_dtype_t weight_dtype, double eps,
    const int64_t* positions, const int64_t positions_shape[3], const int64_t positions_strides[3],
    const double* inv_freq, const int32_t* pair_axes, rope_dtype_t table_dtype, int64_t mode,
    const int64_t partial_slice[2], void* stream);

/*
 * rope_qk_norm_bwd -- its backward pass: dq and dk receive the gradients for q
 * and k, dq_weight and dk_weight (D weight_dtype numbers) those for the
 * weights, summed over every row in fp32 and rounded once; either may be NULL
 * (not computed), and must be where the weight is. q_grad and k_grad are the
 * gradients for q_out and k_out; dq may be q_grad, with its strides, and dk
 * k_grad. Without rows the weights' gradients are 0.
 *
 *   workspace     device buffer of workspace_bytes, 16-byte aligned, at least
 *                 rope_qk_norm_workspace(D); not looked at when neither
 *                 weight's gradient is asked for. Two calls that may run at
 *                 once need one each.
 *   Other arguments and checks as above; the workspace before positions.
 */
ROPE_API rope_status_t rope_qk_norm_bwd(
    int64_t B, int64_t S, rope_dtype_t dtype, const rope_rows_t* dq, const rope_rows_t* dk, void* dq_weight,
    void* dk_weight, const rope_rows_t* q_grad, const rope_rows_t* k_grad, const rope_rows_t* q, const rope_rows_t* k,
    const void* q_weight, const void* k_weight, rope_dtype_t weight_dtype, double eps, const int64_t* positions,
    const int64_t positions_shape[3], const int64_t positions_strides[3], const double* inv_freq,
    const int32_t* pair_axes, rope_dtype_t table_dtype, int64_t mode, const int64_t partial_slice[2], void* workspace,
    int64_t workspace_bytes, void* stream);

/* Bytes of workspace that a rope_qk_norm_bwd with heads of D lanes needs. */
ROPE_API int64_t rope_qk_norm_workspace(int64_t D);

/* ====================== checks and launch plans ====================== */

/*
 * rope_partial_check -- run every argument check of rope_partial_fwd_inplace
 * (either direction: they are the same) and return the status it would
 * return, without launching anything or touching device memory. For callers
 * that validate ahead of time, as the page's graph-mode meta implementation
 * does at compile time (section 调用说明, graph mode). Pointers are only
 * compared with NULL.
 */
ROPE_API rope_status_t rope_partial_check(
    const void* x, const int64_t x_shape[4], rope_dtype_t dtype,
    const void* r1, const int64_t r1_shape[4], const int64_t r1_strides[4],
    const void* r2, const int64_t r2_shape[4], const int64_t r2_strides[4],
    rope_dtype_t table_dtype, int64_t mode, const int64_t partial_slice[2]);

/* Kernels of the launch plan (rope_partial_launch_info). */
#define ROPE_KERNEL_NONE 0   /* no-op call: nothing is launched */
#define ROPE_KERNEL_VECTOR 1 /* 16-byte vector kernel */
#define ROPE_KERNEL_SCALAR 2 /* one thread per pair, 64-bit indexing (2^31 rows or more) */
#define ROPE_KERNEL_ROWS 3   /* one thread per pair, rows of threads, any alignment */
#define ROPE_LAUNCH_INFO_LEN 8

/*
 * rope_partial_launch_info -- the launch plan a call with these arguments
 * would use (either direction: they plan alike), for tests and profiling.
 * Runs the checks of rope_partial_check first and returns their status; on
 * ROPE_OK, info (caller-owned, ROPE_LAUNCH_INFO_LEN elements) receives:
 *   [0] ROPE_KERNEL_NONE, _VECTOR, _ROWS or _SCALAR;
 *   [1] blocks of the launch (0 for the scalar kernel, whose grid follows
 *       the device's compute-unit count at launch);
 *   [2] threads per block;
 *   vector kernel: [3] heads per thread, [4] head lanes per tile, [5] tiles
 *       per block, [6] XCD run length (consecutive blocks kept on one XCD),
 *       [7] 16-byte vectors each row's threads cover;
 *   row kernel: [4] rows per block, [7] threads per row.
 * Entries that do not apply are 0. Launches nothing and touches no memory;
 * pointers are only compared with NULL and checked for alignment.
 * NULL info is ROPE_ERR_NULLPTR.
 */
ROPE_API rope_status_t rope_partial_launch_info(
    const void* x, const int64_t x_shape[4], rope_dtype_t dtype,
    const void* r1, const int64_t r1_shape[4], const int64_t r1_strides[4],
    const void* r2, const int64_t r2_shape[4], const int64_t r2_strides[4],
    rope_dtype_t table_dtype, int64_t mode, const int64_t partial_slice[2],
    int64_t info[ROPE_LAUNCH_INFO_LEN]);

/*
 * rope_partial_launch_info_pos -- the launch plan of an in-place position
 * call (rope_partial_fwd_inplace_pos / _bwd_inplace_pos) with these arguments,
 * for tests and profiling. Runs that call's checks first and returns their
 * status; on ROPE_OK, info (caller-owned, ROPE_LAUNCH_INFO_LEN elements)
 * receives:
 *   [0] ROPE_KERNEL_NONE, _VECTOR, _ROWS or _SCALAR;
 *   [1] blocks of the launch (0 for the scalar kernel);
 *   [2] threads per block;
 *   vector kernel: [3] heads per thread, [4] head lanes per position,
 *       [5] positions per block, [6] head chunks per position, [7] 16-byte
 *       vectors each row's threads cover;
 *   row kernel: [4] rows per block, [7] threads per row.
 * Entries that do not apply are 0. Launches nothing and touches no memory;
 * pointers are only compared with NULL and checked for alignment. NULL
 * info is ROPE_ERR_NULLPTR.
 */
ROPE_API rope_status_t rope_partial_launch_info_pos(
    const void* x, const int64_t x_shape[4], rope_dtype_t dtype,
    const int64_t* positions, const int64_t positions_shape[2], const int64_t positions_strides[2],
    const double* inv_freq, rope_dtype_t table_dtype, int64_t mode, const int64_t partial_slice[2],
    int64_t info[ROPE_LAUNCH_INFO_LEN]);

/*
 * rope_partial_launch_info_axes -- the launch plan of an in-place call with
 * positions on several axes; info as for rope_partial_launch_info_pos.
 */
ROPE_API rope_status_t rope_partial_launch_info_axes(
    const void* x, const int64_t x_shape[4], rope_dtype_t dtype, const int64_t* positions,
    const int64_t positions_shape[3], const int64_t positions_strides[3], const double* inv_freq,
    const int32_t* pair_axes, rope_dtype_t table_dtype, int64_t mode, const int64_t partial_slice[2],
    int64_t info[ROPE_LAUNCH_INFO_LEN]);

/* ===================== projection with a rotary epilogue ===================== */

/*
 * rope_proj_fwd -- a head projection whose epilogue rotates each head's
 * slice before the result is stored: for every token m = b*S + s and output
 * lane n = h*Dh + j,
 *     p[m,n] = fl32( sum_k x[m,k] * w[n,k] )            (fp32 accumulation)
 *     y[b,s,h,j] = p rotated on the lanes [start,end) of each head, forward,
 *                  as rope_partial_fwd_inplace rotates fp32 data, then
 *                  rounded once to y's type.
 * This is the Q projection and RoPE stages of "ascend-transformer-boost 的
 * MlaPreprocessOperation：MLA 预处理四阶段融合算子深度解析", section 3 (the
 * WUQ matmul gives headNum x 192 lanes per token; Q[..., :qRopeDim] is then
 * rotated with cos/sin of shape [tokenNum, 64] given from outside) and
 * section 2 (qRopeDim, qRotaryCoeff), fused so that the projection result is
 * rotated in registers: it is never rounded to the storage type, and never
 * written and read back, before the rotation. The quantisation, RMS norms
 * and KV-cache stages of that page are not part of this call.
 *
 *   y            device buffer of the result, (B, S, H, Dh) contiguous, of
 *                type y_dtype; owned by the caller; must not overlap x or w.
 *   y_dtype      the type of x and w, or ROPE_DTYPE_F32 (no final rounding).
 *   x            device buffer (B*S, K), row-major, of `dtype`.
 *   w            device buffer (H*Dh, K), row-major, of `dtype`: output lanes
 *                by inputs, as a linear layer stores its weight (the page's
 *                transposed-weight default).
 *   dtype        ROPE_DTYPE_BF16 or ROPE_DTYPE_F16.
 *   y_shape      host array {B, S, H, Dh}.
 *   K            inputs per token: a positive multiple of 64.
 *   r1, r2, shapes and strides, table_dtype, mode, partial_slice
 *                as for rope_partial_fwd_inplace, against y's shape: tables
 *                (1 or B, 1 or S, 1 or H, L); the page's case is one row per
 *                token, (B, S, 1, L) or (1, S, 1, L) broadcast over B.
 *   stream       hipStream_t to launch on, or NULL.
 *
 * Checks, in this order: the scalar arguments of rope_partial_fwd_inplace
 * on y's shape with y_dtype (ROPE_ERR_NULLPTR for a NULL y_shape,
 * ROPE_ERR_INVALID otherwise); dtype bf16 or fp16, y_dtype dtype or fp32
 * and K >= 0 (ROPE_ERR_INVALID); an empty y returns ROPE_OK without reading
 * any pointer; K not a positive multiple of 64; Dh not one of 32, 64, 96,
 * 128 and 192 (block tiles of whole heads) nor a multiple of 192 or 128 up
 * to 1024 (a head over whole tiles of 192 or 128 lanes, such as MLA's 576-
 * lane compressed KV with its 64 rope lanes); or, for such a wide head, a
 * rotate_half or coefficient group of the slice (2 x its pair distance
 * lanes) that spans two tiles, unless K is a multiple of 128 and every
 * group lies in one 256-lane column tile of y (ROPE_ERR_UNSUPPORTED);
 * NULL y, x or w (ROPE_ERR_NULLPTR); y, x or w not 16-byte aligned or
 * sizes beyond 64-bit offsets (ROPE_ERR_INVALID); x or w of 2^31 elements
 * or more (ROPE_ERR_UNSUPPORTED); y overlapping x or w (ROPE_ERR_INVALID); then,
 * for a non-empty slice, the tables as for rope_partial_fwd_inplace; a grid
 * too large for one launch (ROPE_ERR_UNSUPPORTED); finally the launch
 * (ROPE_ERR_RUNTIME). An empty slice gives the plain projection. The
 * library allocates nothing; results are deterministic (each output is
 * accumulated by one wave in a fixed order).
 */
ROPE_API rope_status_t rope_proj_fwd(
    void* y, rope_dtype_t y_dtype, const void* x, const void* w, rope_dtype_t dtype,
    const int64_t y_shape[4], int64_t K,
    const void* r1, const int64_t r1_shape[4], const int64_t r1_strides[4],
    const void* r2, const int64_t r2_shape[4], const int64_t r2_strides[4],
    rope_dtype_t table_dtype, int64_t mode, const int64_t partial_slice[2],
    void* stream);

/*
 * Low-rank adapters of many requests beside one shared projection: `count`
 * adapters of `rank`, and the adapter of each token.
 */
typedef struct rope_lora {
    const void* a;            /* device (count, rank, K), of x's type: the products with x */
    const void* b;            /* device (count, H*Dh, rank), of x's type: their products to output lanes */
    const int32_t* adapters;  /* device (B*S): the adapter of each token; outside [0, count): none */
    const float* scales;      /* device (count), or NULL: 1 */
    int64_t count, rank;      /* rank: a multiple of 8, at most ROPE_LORA_RANK_MAX; count 0: no adapters */
} rope_lora_t;

#define ROPE_LORA_RANK_MAX 128

/*
 * rope_proj_lora_fwd -- rope_proj_fwd with the token's own low-rank adapter:
 * for token m with adapter i = adapters[m],
 *     h[m,r] = scales[i] * fl32( sum_k x[m,k] * a[i,r,k] )
 *     p[m,n] = fl32( sum_k x[m,k] * w[n,k]  +  sum_r h[m,r] * b[i,n,r] )
 *     y[b,s,h,j] = p rotated on the lanes [start,end) of each head, then
 *                  rounded once to y's type.
 * h is kept in fp32 (16-bit outputs may take it as the sum of two values of
 * 8 bits each, fp32 outputs of three: the part left out is below 2^-16 and
 * 2^-24 of it). A token without an adapter gives rope_proj_fwd's result up to
 * the order of summation. Tokens may have their adapters in any order (calls
 * of many tokens sort them); up to 1023 adapters are fastest. A token whose h
 * or whose adapter is not finite may get NaN where an infinity would be exact;
 * no other token's result changes.
 *
 *   workspace        device buffer of workspace_bytes, 16-byte aligned, used
 *                    during the call: at least
 *                    rope_proj_lora_workspace(y_shape, K, rank). Two calls
 *                    that may run at once need one each.
 *   Other arguments are those of rope_proj_fwd, and so are the shapes it
 *   takes, except that a slice's rotation groups may lie anywhere in a head.
 *
 * Checks: rope_proj_fwd's in their order, with these after the sizes of x
 * and w: a NULL lora (ROPE_ERR_NULLPTR); count or rank negative, rank not a
 * multiple of 8 (ROPE_ERR_INVALID) or above ROPE_LORA_RANK_MAX
 * (ROPE_ERR_UNSUPPORTED), count or rank 0 is a projection without adapters;
 * NULL a, b, adapters or workspace; a, b or workspace not 16-byte aligned,
 * sizes beyond 64 bits, too small a workspace, y overlapping a, b, adapters,
 * scales or the workspace, the workspace overlapping any input (ROPE_ERR_INVALID;
 * of a larger workspace only the bytes it has to hold count); and, after the
 * tables' own checks, y or the workspace overlapping a table.
 * Asynchronous on `stream`; nothing is allocated; deterministic.
 */
ROPE_API rope_status_t rope_proj_lora_fwd(
    void* y, rope_dtype_t y_dtype, const void* x, const void* w, rope_dtype_t dtype,
    const int64_t y_shape[4], int64_t K, const rope_lora_t* lora,
    const void* r1, const int64_t r1_shape[4], const int64_t r1_strides[4],
    const void* r2, const int64_t r2_shape[4], const int64_t r2_strides[4],
    rope_dtype_t table_dtype, int64_t mode, const int64_t partial_slice[2],
    void* workspace, int64_t workspace_bytes, void* stream);

/* Bytes of workspace that a rope_proj_lora_fwd of this shape needs (0 when
 * nothing is computed or the arguments are out of range). */
ROPE_API int64_t rope_proj_lora_workspace(const int64_t y_shape[4], int64_t K, int64_t rank);

/* Kernels of a projection's launch plan (rope_proj_launch_info). */
#define ROPE_KERNEL_PROJ_HEADS 4  /* tiles of whole heads: 384 x 192 (12 waves) or 256 x 128 (8 waves) */
#define ROPE_KERNEL_PROJ_SQUARE 5 /* 256 x 256 tiles, 4 waves of 128 x 128 */

/*
 * rope_proj_launch_info -- the launch plan rope_proj_fwd would use for
 * these arguments (y, x and w themselves aside), for tests and profiling.
 * Runs rope_proj_fwd's checks, with stand-ins for the y, x and w pointers
 * that pass the NULL, alignment and overlap checks, and returns their
 * status; on ROPE_OK, info (caller-owned, ROPE_LAUNCH_INFO_LEN elements)
 * receives:
 *   [0] ROPE_KERNEL_NONE (an empty y), ROPE_KERNEL_PROJ_HEADS or
 *       ROPE_KERNEL_PROJ_SQUARE (K a multiple of 128 and every rotation
 *       group of the slice inside one 256-lane column tile);
 *   [1] blocks; [2] threads per block; [3] tokens and [4] output lanes per
 *       block tile;
 *   square tiles: [5] the epilogue: 0 the general one (any geometry), 1 the
 *       vector epilogue with rotation partners in the 8-lane vector
 *       (interleave, or no slice), 2 the vector epilogue with partners whole
 *       vectors away inside one wave's 128 lanes; [6] 1 when the tables' rows
 *       are staged in LDS during the K loop (both tables shared by all heads,
 *       a row of L values 16, 32, 64 or 128 bytes).
 * Entries that do not apply are 0. Launches nothing and touches no memory;
 * table pointers are only compared with NULL and checked for alignment.
 * NULL info is ROPE_ERR_NULLPTR.
 */
ROPE_API rope_status_t rope_proj_launch_info(
    rope_dtype_t y_dtype, rope_dtype_t dtype, const int64_t y_shape[4], int64_t K,
    const void* r1, const int64_t r1_shape[4], const int64_t r1_strides[4],
    const void* r2, const int64_t r2_shape[4], const int64_t r2_strides[4],
    rope_dtype_t table_dtype, int64_t mode, const int64_t partial_slice[2],
    int64_t info[ROPE_LAUNCH_INFO_LEN]);

/* Kernels of a projection with adapters beside its tiles (rope_proj_lora_launch_info). */
#define ROPE_KERNEL_PROJ_FEW 6     /* units of 32 output lanes by up to 64 tokens, unsorted */
#define ROPE_KERNEL_PROJ_GENERAL 7 /* 16 tokens of one head, any slice, unsorted */

/*
 * rope_proj_lora_launch_info -- the launch plan rope_proj_lora_fwd would use
 * for these arguments and `count` adapters of `rank`, for tests and profiling:
 * as rope_proj_launch_info, with stand-ins for the adapters' pointers and the
 * workspace too. info[0] ROPE_KERNEL_NONE, ROPE_KERNEL_PROJ_HEADS, _SQUARE,
 * _FEW or _GENERAL; [1] to [6] as there ([1] a bound on the blocks with work
 * where tokens are sorted); [7] 1 when the tokens are sorted by adapter first.
 */
ROPE_API rope_status_t rope_proj_lora_launch_info(
    rope_dtype_t y_dtype, rope_dtype_t dtype, const int64_t y_shape[4], int64_t K, int64_t count, int64_t rank,
    const void* r1, const int64_t r1_shape[4], const int64_t r1_strides[4],
    const void* r2, const int64_t r2_shape[4], const int64_t r2_strides[4],
    rope_dtype_t table_dtype, int64_t mode, const int64_t partial_slice[2],
    int64_t info[ROPE_LAUNCH_INFO_LEN]);

/* ============================== status ============================== */

/* Static text for a status code; never NULL. */
ROPE_API const char* rope_status_string(rope_status_t status);

/* Text describing the last non-OK status returned on the calling thread
 * (which check failed, or the HIP error); "" if none. The pointer stays valid
 * until the next call on that thread. */
ROPE_API const char* rope_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* ROPE_PARTIAL_H */
