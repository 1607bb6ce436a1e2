/*
 * rc.h -- C ABI of the write-time FP8 ring KV cache for one GB300 (sm_103a).
 *
 * The operations come from the pages about "Runway Characters: Serving a 57B
 * Video Diffusion Transformer for Real-Time Conversation" (arXiv 2611.05642):
 *   - paperdot abstract mirror: the cache is a ring; keys get RoPE and FP8
 *     quantisation a single time, when written; a reset of the positions
 *     rotates the stored keys by the difference.  A chunk's 240 attention
 *     calls each read 5,788 slots, 757 of them new.
 *   - cpdf.ai blog, section "Como rodar 57B em tempo real com batch size 1":
 *     rotary positions and FP8 quantisation move from read time to write
 *     time, and the ring advances the window without copies.
 *   - cpdf.ai blog, section "Blackwell, escalabilidade e limites do
 *     decodificador": the FP8 attention kernel uses per-head scales.
 *
 * Conventions shared by every call:
 *   - Status: 0 (RC_OK) or a negative RC_ERR_* code.  Argument and state
 *     errors are found on the host before anything is launched, and leave the
 *     cache unchanged.  Errors of kernels already launched surface as
 *     RC_ERR_CUDA from a later call, or from rc_cache_sync.  No C++ exception
 *     crosses this boundary.
 *   - Device pointers are plain CUDA device addresses (for example a torch
 *     tensor's data_ptr()), 16-byte aligned (RC_ERR_ARG otherwise).  The
 *     caller keeps them alive until the work on `stream` that reads or
 *     writes them has finished.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *     stream).  Calls on one handle must be issued on one stream, or ordered
 *     by the caller; a handle is not thread-safe.
 *   - Memory: rc_cache_create allocates every device and pinned host buffer
 *     the handle will ever use.  No later call allocates, for any write size
 *     up to max_write.
 *   - Layouts: K, V and Q are bf16, token-major [n][heads][head_dim] with
 *     head_dim contiguous.  The attention output is fp32 with the same layout.
 *     head_dim is 64 or 128.
 *   - CUDA graphs: rc_cache_write, rc_attend and rc_cache_delta_rotate only
 *     launch kernels on `stream` once each has been called directly on the
 *     device (the first call sets kernel attributes), so a run of them can be
 *     captured into a graph.  A write to capture must have consecutive
 *     positions (p0, p0 + 1, ...) or repeat the positions of a recent write:
 *     any other position vector goes to the device through a pinned buffer
 *     guarded by an event, which a capture cannot hold.  The host-side
 *     bookkeeping (slots, write groups, the positions the next attention
 *     rotates its queries at) is done when a call is captured, and the graph
 *     keeps that call's arguments: launch each captured graph once, in the
 *     order of capture, with no direct call on the handle in between.
 */
#ifndef RC_H
#define RC_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes ------------------------------------------------------ */
#define RC_OK 0
#define RC_ERR_ARG (-1)         /* bad argument: null pointer, size or index out of range,
                                   two tokens of one write on the same slot */
#define RC_ERR_STATE (-2)       /* call not valid in the current state: attention on a
                                   layer never written, or query count different from
                                   that layer's last write */
#define RC_ERR_CUDA (-3)        /* a CUDA runtime call or a launched kernel failed */
#define RC_ERR_OOM (-4)         /* rc_cache_create could not allocate */
#define RC_ERR_TIMEOUT (-5)     /* a kernel gave up a bounded wait and returned early;
                                   its output is not valid */
#define RC_ERR_UNSUPPORTED (-6) /* shape not supported (head_dim other than 64 or 128,
                                   or a device that is not sm_103) */
#define RC_ERR_BOUNDS (-7)      /* bounds-checked build only (rc_build_flags): a kernel's
                                   index check failed and the access was skipped, or a
                                   buffer's guard bytes were overwritten; results are
                                   not valid */

/* ---- configuration ------------------------------------------------------ */
/* Keep the unrotated bf16 K, V of every slot as well, so that rc_attend_readtime
   can redo RoPE and quantisation of the whole cache at read time. */
#define RC_F_READTIME_ABLATION 1u
/* Allocate a second bank of rings so that rc_cache_window_shift can move the
   stored tokens the way a concatenating cache would (the copy-based window
   ablation; doubles the ring memory; not combinable with the flag above). */
#define RC_F_COPY_WINDOW 2u
/* A 16-bit ring instead of E4M3 + per-slot scales: the non-FP8 cache of the
   comparison in the cpdf.ai blog, section "Blackwell, escalabilidade e
   limites do decodificador" (FP8 saves time on H100 and costs time on B200
   without an FP8 attention kernel).  Writes round RoPE(K) once to bf16 and
   store V converted once to fp16 (exact for 2^-17 <= |v| < 65520 and zero;
   smaller magnitudes round to fp16's subnormal step, larger ones become
   +-inf); delta rotations re-rotate every stored key and round it back to
   bf16; attention computes softmax(Q K^T / sqrt(d)) V with fp32 accumulation.
   Doubles the ring memory, keeps no scales; rc_cache_export_bf16 replaces
   rc_cache_export.  Not combinable with the two flags above. */
#define RC_F_BF16_CACHE 4u

typedef struct rc_config {
    int layers;       /* attention layers with one ring each (>= 1) */
    int heads;        /* heads per layer (>= 1) */
    int head_dim;     /* 64 or 128 */
    int slots;        /* ring capacity C per layer (>= 1) */
    int max_write;    /* largest n of one write (1 .. slots) */
    double rope_base; /* RoPE base; theta_i = base^(-2i/head_dim) (> 1) */
    unsigned flags;   /* RC_F_* */
} rc_config;

typedef struct rc_cache rc_cache; /* opaque; owns all of its memory */

/*
 * Create a cache on CUDA device `device` and store the handle in *out.
 * Every slot starts empty.  Allocates the FP8 rings (2 * layers * heads *
 * ceil(slots/128)*128 * head_dim bytes), the per-slot scales, the RoPE table
 * pool and the pinned position staging, and with RC_F_READTIME_ABLATION the
 * bf16 store.  On error *out is NULL and nothing is leaked.
 */
int rc_cache_create(const rc_config *cfg, int device, rc_cache **out);

/*
 * Write n new tokens into ring `layer` (paperdot abstract: RoPE and FP8
 * quantisation happen here, a single time per token).  K_bf16 and V_bf16 are device
 * pointers to [n][heads][head_dim] bf16.  positions is a HOST array of n
 * int64 token positions (any sign).  Token t goes to slot
 * floormod(positions[t] - delta_total, slots), replacing what was there.
 * For every head, K is rotated by RoPE at its position; then K and V each get
 * one fp32 scale s = fl32(amax/448) over the n tokens of that head (s = 1 if
 * amax = 0), and each element is stored as the E4M3 code of fl32(x/s),
 * rounded to nearest even and saturated to +-448.
 * Errors: RC_ERR_ARG if layer is out of range, n < 1 or n > max_write, a
 * pointer is NULL, or two tokens map to one slot.
 * A position vector that is not an arithmetic run p0, p0+1, ... is copied to
 * the device through pinned staging; an arithmetic run needs no copy.
 */
int rc_cache_write(rc_cache *h, int layer, const void *K_bf16, const void *V_bf16,
                   const int64_t *positions, int n, void *stream);

/*
 * Position reset (paperdot abstract: resetting the positions rotates the
 * stored keys by the difference).  Every occupied slot of every layer moves from position p to
 * p + delta without moving slots: the stored keys are dequantised, rotated
 * by delta, and each (layer, head, write group) is requantised in place with
 * a fresh scale from its new amax.  Values are untouched.  The layers' last
 * write positions move by delta too.  delta = 0 is a no-op.
 */
int rc_cache_delta_rotate(rc_cache *h, int64_t delta, void *stream);

/*
 * The copy-based window, an ablation of the ring (paperdot abstract: the
 * window advances "without copies"; this is the copy).  A cache that keeps
 * its tokens in position order moves them k slots down when k new positions
 * arrive, then writes the new tokens at the end.  This call does that move in
 * every layer: slot s takes what slot (s + k) mod slots held (K and V codes,
 * their scales and write groups, one read and one write of every ring, into
 * the second bank), and from then on a token at position p lives in slot
 * floormod(p - delta_total - (sum of shifts), slots).  The set of stored
 * tokens, their codes and every attention result are those of the ring;
 * rc_cache_export returns the slots in their shifted order.  k = 0 (or a
 * multiple of slots) moves nothing.
 * Errors: RC_ERR_STATE unless the cache was created with RC_F_COPY_WINDOW;
 * RC_ERR_ARG for a NULL handle or k < 0.
 */
int rc_cache_window_shift(rc_cache *h, int64_t k, void *stream);

/*
 * Attention call (paperdot abstract: the new tokens' queries read the whole
 * cache).  Q_bf16 is a device pointer to [n][heads][head_dim] bf16 queries of
 * the layer's last write; each is rotated at that token's (current) position.
 * out_f32 is a device pointer to [n][heads][head_dim] fp32:
 *   out = softmax(q . k_j / sqrt(head_dim)) over the occupied slots j, times v_j,
 * with k_j, v_j the stored codes times their slot's scale.  No mask.
 * Errors: RC_ERR_STATE if the layer was never written or n differs from the
 * layer's last write; RC_ERR_ARG for NULL pointers or a bad layer.
 */
int rc_attend(rc_cache *h, int layer, const void *Q_bf16, float *out_f32, int n,
              void *stream);

/*
 * Read-time ablation of rc_attend (the original design the pages describe
 * in the abstract and in the cpdf.ai section "Como rodar 57B em tempo real
 * com batch size 1": RoPE and FP8 quantisation of the WHOLE cache redone in
 * every attention call).  Rebuilds this layer's FP8 ring from the unrotated
 * bf16 store into a scratch ring, then runs the same attention kernel on it.
 * Every stored key is rotated at its slot's CURRENT position: the store keeps
 * each slot's position on the device and rc_cache_delta_rotate moves it, so
 * after any number of resets the read-time ring holds the keys the write-time
 * ring would hold had it been written at today's positions.  Each call first
 * rebuilds the angle table of all slots (fp64 angles) from those positions.
 * Requires RC_F_READTIME_ABLATION, else RC_ERR_STATE.  The read-time ring
 * quantises each head with ONE scale over all occupied slots (per K and V),
 * so its codes differ from the write-time ring's wherever that ring holds
 * several write groups with different scales; the rotated keys before
 * quantisation are the same.
 */
int rc_attend_readtime(rc_cache *h, int layer, const void *Q_bf16, float *out_f32,
                       int n, void *stream);

/* Free everything the handle owns (waits for its device work first). NULL is ignored. */
void rc_cache_destroy(rc_cache *h);

/* A static description of a status code. */
const char *rc_status_string(int status);

/* ---- inspection and test support -------------------------------------- */

/* Synchronise the handle's last stream and report any kernel error or timeout
   (RC_ERR_TIMEOUT), and in the bounds-checked build a failed index check or
   overwritten guard bytes (RC_ERR_BOUNDS).  The device status word is cleared. */
int rc_cache_sync(rc_cache *h);

/* How this library was built: RC_BUILD_BOUNDS_CHECK is set in the bounds-
   checked build (librc_bounds.so, compiled with -DRC_BOUNDS_CHECK).  There,
   the write, rotation, read-time and attention kernels test the index of each global
   access they make against the buffer it addresses before making it (a
   failure skips the access and records the site; nothing traps), and every
   device buffer of a handle sits between two 256-byte guard zones filled with
   0xA5 that rc_cache_sync checks.  The normal build has neither and returns 0.
   Needs no device. */
#define RC_BUILD_BOUNDS_CHECK 1u
unsigned rc_build_flags(void);

/*
 * Failure-path support.  Every wait inside the attention kernel is bounded:
 * past `ns` nanoseconds (default 2 s) the kernel gives up, records where, frees
 * its tensor memory and returns, and the next rc_cache_sync reports
 * RC_ERR_TIMEOUT (and clears the record; the ring itself is not modified by an
 * attention call, so the handle stays usable).  ns = 0 gives up on any wait
 * whose phase is not already complete, which makes a wait run out on purpose.
 * Errors: RC_ERR_ARG for a NULL handle or ns above 60 s.
 *
 * Host-side fault injection, read from the environment at each use:
 * RC_FAULT_INJECT=alloc:K makes the K-th allocation (1-based, device or
 * pinned) of rc_cache_create fail, which then returns RC_ERR_OOM having freed
 * everything it had allocated; RC_FAULT_INJECT=launch makes every call that
 * launches kernels return RC_ERR_CUDA after its argument checks, before it
 * changes anything.
 */
int rc_cache_set_wait_limit(rc_cache *h, uint64_t ns);

/*
 * Write n new tokens into ring `layer` straight from the K/V projection: the
 * write fused into the projection's FP8 GEMM (the single-GPU half of the
 * pages' fused FP8 GEMM: paperdot abstract; cpdf.ai blog, "Como rodar 57B em
 * tempo real com batch size 1").  With X, Wk, Wv E4M3 codes and one scale
 * each,
 *   K[t][h][i] = x_scale * wk_scale * sum_k X[t][k] * Wk[h*head_dim + i][k]
 * and V likewise with Wv, wv_scale, computed on the tensor cores (fp32
 * accumulation); then written as rc_cache_write writes its K and V (RoPE at
 * positions[t], one scale per head for K and for V, E4M3 codes into the
 * slots), from the fp32 products with no bf16 rounding in between.
 * X: device [n][hidden] uint8, row stride hidden bytes; Wk, Wv: device
 * [heads*head_dim][hidden] uint8 (one weight row per output feature); all
 * 16-byte aligned.  hidden: a multiple of 64.  positions: HOST int64 [n], as
 * for rc_cache_write.  Stream-ordered; the caller keeps X, Wk, Wv alive until
 * the work on `stream` has finished.
 * A fused write whose kernel gave up a bounded wait (rc_cache_sync then reports
 * RC_ERR_TIMEOUT) leaves its slots undefined; writing them again repairs them.
 * Errors: RC_ERR_ARG (a pointer NULL or unaligned, layer out of range, n < 1,
 * n > max_write or n > 2048, hidden not a positive multiple of 64, a scale not
 * positive, two tokens on one slot); RC_ERR_UNSUPPORTED with RC_F_BF16_CACHE
 * or RC_F_READTIME_ABLATION (the read-time store keeps bf16 K and V, which
 * this path never forms).
 */
int rc_cache_write_fused(rc_cache *h, int layer, const uint8_t *X, float x_scale,
                         const uint8_t *Wk, float wk_scale, const uint8_t *Wv, float wv_scale,
                         int hidden, const int64_t *positions, int n, void *stream);

/*
 * Copy ring `layer` to HOST buffers in canonical layout (synchronous):
 * kcodes, vcodes: uint8 [heads][slots][head_dim] E4M3 codes; kscale, vscale:
 * fp32 [heads][slots]; pos: int64 [slots] position (INT64_MIN = empty);
 * gid: int64 [slots] serial number of the write that filled the slot
 * (INT64_MIN = empty; writes are numbered 0, 1, ... per handle).  Any
 * pointer may be NULL to skip that table.
 */
int rc_cache_export(rc_cache *h, int layer, uint8_t *kcodes, float *kscale,
                    uint8_t *vcodes, float *vscale, int64_t *pos, int64_t *gid);

/*
 * Copy the scratch ring that the last rc_attend_readtime call built (same
 * canonical layouts as rc_cache_export; synchronous).  RC_ERR_STATE without
 * RC_F_READTIME_ABLATION.
 */
int rc_cache_export_readtime(rc_cache *h, uint8_t *kcodes, float *kscale,
                             uint8_t *vcodes, float *vscale);

/*
 * Copy ring `layer` of a RC_F_BF16_CACHE cache to HOST buffers (synchronous):
 * kbits, vbits: uint16 [heads][slots][head_dim] bf16 bit patterns (RoPE'd keys
 * at their current positions; the stored fp16 values rounded to bf16, which
 * returns each in-range value as written; zeros in empty slots); pos,
 * gid as in rc_cache_export.  Any pointer may be NULL.  RC_ERR_STATE without
 * the flag (and rc_cache_export answers RC_ERR_STATE with it).
 */
int rc_cache_export_bf16(rc_cache *h, int layer, uint16_t *kbits, uint16_t *vbits,
                         int64_t *pos, int64_t *gid);

/* ---- allocation-free write into a caller-owned ring -------------------- */
/*
 * No counterpart in the paper: this is an integration convenience.
 *
 * Some callers cannot call cudaMalloc: a process whose device memory is all
 * reserved up front by another allocator (a framework's caching allocator or
 * a fixed arena), where a new allocation would fail or fragment that pool; or
 * a latency-critical loop that must never pay for cudaMalloc / cudaFree, which
 * can synchronise the whole device.  rc_ring_write_noalloc serves them: it
 * performs exactly the write of rc_cache_write (RoPE table kernel, then the
 * fused RoPE + per-head amax + E4M3 write kernel) into ring buffers that the
 * CALLER owns, and it allocates nothing.  Its only scratch -- a copy of
 * non-arithmetic positions and the per-token cos/sin table -- lives in one
 * file-scope __device__ array of about 2 MiB (RC_NOALLOC_MAX_TOKENS tokens x
 * 64 pairs x 8 bytes, plus 32 KiB), which every GPU that loads the library
 * holds until the process exits.  The RoPE frequencies go to the kernel as
 * parameters.
 *
 * Rules:
 *   - n <= RC_NOALLOC_MAX_TOKENS, else RC_ERR_ARG (nothing is launched).
 *   - The first call on a device looks up the array's device address on the
 *     current device (cudaGetSymbolAddress) and keeps it; make that first call
 *     before any stream capture.  Resetting that device (cudaDeviceReset)
 *     afterwards is not supported: the kept address would be stale.
 *   - Every call on a device shares the one array, and it keeps the last
 *     call's contents.  Calls that overlap on the GPU (other streams or
 *     threads without ordering) race on it; order them on one stream.
 *   - positions is a HOST array.  An arithmetic run p0, p0+1, ... needs no
 *     copy; any other position vector is copied into the array from the
 *     caller's (pageable) memory with cudaMemcpyAsync, which returns once the
 *     bytes are staged.
 *   - The caller keeps the ring state: delta_total (the sum of resets applied
 *     to this ring) and a write-group index in [0, slots) unique among the
 *     ring's live groups.  There is no delta rotation or attention entry on a
 *     caller-owned ring; this is the write alone.
 *
 * Ring layout (T = ceil(slots / 128) tiles per head, Cpad = 128 T), all device
 * memory the caller allocated:
 *   kcodes [heads][T][128][head_dim] E4M3: slot s is row s % 128 of tile
 *          s / 128; byte d of a row sits at 16-byte chunk (d / 16) XOR x,
 *          x = row % 8 (head_dim 128) or (row / 2) % 4 (head_dim 64).
 *   vcodes [heads][T][head_dim][128] E4M3 (transposed): element (d, s) sits in
 *          row d of tile s / 128 at chunk ((s % 128) / 16) XOR (d % 8).
 *   kscale, vscale [heads][Cpad] fp32: the scale of each slot's write group.
 *   group  [Cpad] int32: the slot's write-group index (-1 = empty).
 */
#define RC_NOALLOC_MAX_TOKENS 4096

typedef struct rc_ring_view {
    uint8_t *kcodes;  /* device, see the layout above */
    uint8_t *vcodes;
    float *kscale;
    float *vscale;
    int32_t *group;
    int heads;        /* >= 1 */
    int head_dim;     /* 64 or 128 */
    int slots;        /* ring capacity C >= 1 */
} rc_ring_view;

int rc_ring_write_noalloc(const rc_ring_view *ring, const void *K_bf16, const void *V_bf16,
                          const int64_t *positions, int n, int64_t delta_total,
                          int32_t group, double rope_base, void *stream);

/* ---- positions with several axes ---------------------------------------- */
/*
 * Rotary positions for tokens that have a place on several axes (time, height,
 * width of a video; one axis for text).  The head_dim / 2 dimension pairs
 * (2i, 2i + 1) are divided among the axes in order: the first sections[0] pairs
 * turn by the token's position on axis 0, the next sections[1] by axis 1, and
 * so on.  Pair number r of an axis with w pairs has the frequency
 * base^(-r / w) (an axis is a rotary embedding of its own, of 2 w dims); with
 * RC_ROPE_SHARED_FREQS pair i of the head keeps base^(-2i / head_dim) whatever
 * its axis.  One axis with head_dim / 2 pairs is the RoPE of rc_cache_write.
 *
 * A plan holds each pair's axis and its frequency in turns as a 64-bit fixed
 * point fraction, so that position * frequency mod 1 turn is exact integer
 * arithmetic at every int32 position.  It is plain host data: fill it once,
 * keep it by value, pass it to any number of calls.
 */
#define RC_ROPE_SHARED_FREQS 1u
#define RC_ROPE_MAX_AXES 4

typedef struct rc_rope_plan {
    int head_dim;        /* 64 or 128 */
    int axes;            /* 1 .. RC_ROPE_MAX_AXES */
    uint64_t turns[64];  /* pair i: round(frequency / 2 pi * 2^64) */
    uint8_t axis[64];    /* pair i: its axis */
} rc_rope_plan;

/*
 * Fill *plan.  Host only.  Errors: RC_ERR_ARG for a NULL pointer, axes outside
 * 1 .. 4, a section < 0, sections that do not add up to head_dim / 2, base
 * not in (1, 1e9], unknown flags; RC_ERR_UNSUPPORTED for head_dim other than 64 or 128.
 */
int rc_rope_plan_init(rc_rope_plan *plan, int head_dim, int axes, const int *sections, double base,
                      unsigned flags);

#define RC_BF16 0
#define RC_F32 1

/*
 * out[t][h] = x[t][h] turned at token t's positions (inverse = 0), or turned
 * back (inverse = 1: also the gradient of the turn, dx from dout).  x, out:
 * device [n][heads][head_dim] of dtype RC_BF16 or RC_F32, tokens x_stride /
 * out_stride elements apart (>= heads * head_dim, a multiple of 16 bytes), so
 * a slice of a fused projection's rows can be passed.  out may be x (the same
 * address and stride) or lie between its rows, but share no element with it
 * otherwise.  positions: device int32 [axes][n], axes pos_stride elements apart
 * (>= n).  The arithmetic is fp32, rounded once to dtype.  n = 0 does nothing.
 * Errors: RC_ERR_ARG (NULL or unaligned pointers, n < 0, heads < 1, a stride
 * too small or unaligned, out overlapping x, a plan that rc_rope_plan_init did not fill).
 */
int rc_rope_axes(const rc_rope_plan *plan, const void *x, int64_t x_stride, void *out, int64_t out_stride,
                 int dtype, int64_t n, int heads, const int32_t *positions, int64_t pos_stride, int inverse,
                 void *stream);

/* ---- rotary positions in other forms ---------------------------------------- */
/*
 * Forms of rotary embeddings beside the one above: the turned pairs
 * are neighbours or lie half a part apart, a part of the head turns, frequencies
 * are stretched for contexts longer than a model was trained for, and what is
 * turned is multiplied by a gain.  Dims first .. first + dims - 1 of a head turn,
 * the others are copied.  Pair i < dims / 2 is
 *   RC_ROPE_PAIRS    (first + 2i, first + 2i + 1)
 *   RC_ROPE_HALVES   (first + i, first + i + dims / 2)
 * and turns by the token's position on its axis: the first sections[0] pairs by
 * axis 0, and so on.  Pair number r of an axis with w pairs has the frequency
 * theta = base^(-r / w), with RC_ROPE_SHARED_FREQS base^(-2i / dims) (w = dims / 2
 * and r = i below), which `scaling` stretches by `factor` >= 1:
 *   RC_ROPE_SCALE_NONE    not (factor is not read)
 *   RC_ROPE_SCALE_LINEAR  theta / factor (positions divided by factor)
 *   RC_ROPE_SCALE_BASE    base times factor^(w / (w - 1)): the slowest pair's
 *                         frequency is divided by factor, the fastest one's kept
 *   RC_ROPE_SCALE_PARTS   theta (k + (1 - k) / factor), where k goes from 0 to 1
 *                         as the pair's turns in `context` positions,
 *                         context theta / 2 pi, go from low to high
 * A model has to be run with the frequencies that it was trained with: those that
 * go from stretched to kept evenly over the pairs' NUMBERS (between two pairs that
 * turns give, rounded or not) differ from RC_ROPE_SCALE_PARTS by tens of percent
 * for some pairs, and neither they nor a table of factors for each pair are among
 * these forms.
 * One token at one axis with RC_ROPE_PAIRS, the whole head and a gain of 1 is
 * what rc_rope_axes does.
 */
#define RC_ROPE_PAIRS 0
#define RC_ROPE_HALVES 1
#define RC_ROPE_SCALE_NONE 0
#define RC_ROPE_SCALE_LINEAR 1
#define RC_ROPE_SCALE_BASE 2
#define RC_ROPE_SCALE_PARTS 3
#define RC_ROPE_MAX_HEAD_DIM 256

typedef struct rc_rope_spec {
    int head_dim;      /* a multiple of 8, 8 .. RC_ROPE_MAX_HEAD_DIM */
    int first, dims;   /* the part that turns: both even, dims >= 2, first + dims <= head_dim */
    int layout;        /* RC_ROPE_PAIRS or RC_ROPE_HALVES */
    int axes;          /* 1 .. RC_ROPE_MAX_AXES */
    int sections[RC_ROPE_MAX_AXES]; /* pairs of each axis, dims / 2 in all */
    unsigned flags;    /* RC_ROPE_SHARED_FREQS */
    double base;       /* in (1, 1e9] */
    int scaling;       /* RC_ROPE_SCALE_* */
    double factor;     /* 1 .. 1e6 */
    double context;    /* RC_ROPE_SCALE_PARTS: > 0, at most 2^31 */
    double low, high;  /* RC_ROPE_SCALE_PARTS: 0 <= low < high, at most 2^31 */
    float gain;        /* 2^-16 .. 16 */
} rc_rope_spec;

/* What the calls take: plain host data, filled once by rc_rope_form_init. */
typedef struct rc_rope_form {
    int head_dim, first, dims, layout, axes;
    float gain;
    uint64_t turns[RC_ROPE_MAX_HEAD_DIM / 2]; /* pair i: round(frequency / 2 pi * 2^64) */
    uint8_t axis[RC_ROPE_MAX_HEAD_DIM / 2];   /* pair i: its axis */
} rc_rope_form;

/*
 * Fill *form.  Host only.  Errors: RC_ERR_ARG for a NULL pointer and for what is
 * out of the ranges above; RC_ERR_UNSUPPORTED for a head_dim that is no multiple of 8
 * or not in 8 .. RC_ROPE_MAX_HEAD_DIM.
 */
int rc_rope_form_init(rc_rope_form *form, const rc_rope_spec *spec);

/*
 * out[t][h] = gain * (x[t][h] turned at token t's positions) in the part that
 * turns, x[t][h] elsewhere; with back != 0 turned back instead, with the same gain:
 * the gradient, dx from dout.  The other arguments, the arithmetic and the
 * errors are those of rc_rope_axes (its head_dim is the form's).
 */
int rc_rope_turn(const rc_rope_form *form, const void *x, int64_t x_stride, void *out, int64_t out_stride,
                 int dtype, int64_t n, int heads, const int32_t *positions, int64_t pos_stride, int back,
                 void *stream);

/* ---- the paged cache ------------------------------------------------------ */
/*
 * One layer's FP8 cache for many sequences, in pages the CALLER owns (as with
 * rc_ring_write_noalloc, nothing here allocates): any page can serve any
 * sequence, and sequences may share pages they only read.
 *
 * Pages (P = page_tokens: 16, 32, 64 or 128), device memory, 16-byte aligned:
 *   kcodes [pages][kv_heads][P][head_dim]  E4M3 codes
 *   vcodes [pages][kv_heads][head_dim][P]  E4M3 codes (V transposed)
 *   kscale, vscale [pages][kv_heads][P]    E8M0: byte b stands for 2^(b - 127)
 * Each token and head has one scale for K and one for V: the smallest power of
 * two s with max |x| <= 448 s (s = 1 for a row of zeros; s between 2^-124 and
 * 2^7, so magnitudes over 57,344 saturate).  Code times scale is then an exact
 * bf16 number.  A row that holds an infinity or a NaN gets scale byte 255 and
 * zero codes, which read as NaN.  Scale bytes under 3 and 135 .. 254 are not
 * produced; tokens that have them read as some number, infinity or NaN.
 *
 * Metadata of a call (rc_paged_batch), device int32, read when the kernels run,
 * so a captured graph follows the values that are there at each replay:
 *   page_table [seqs][table_pages]  entry i of a row: the page of the
 *       sequence's tokens [i P, i P + P); entries past its length are not read
 *   kv_len [seqs]   tokens of the sequence in the cache, its new ones included
 *   q_start [seqs + 1]  sequence s owns rows q_start[s] .. q_start[s + 1] - 1
 *       of the token-major tensors; its n new tokens are the last n of its
 *       kv_len.  Rows outside every sequence are not touched.
 * max_new and max_kv (host) bound every sequence's n and kv_len; tokens (host) is the
 * row count of the tensors.  They size the launches for the largest sequence: where
 * that takes more than 2^31 - 1 blocks (seqs x max_new / 16 of a write, seqs x
 * kv_heads x a KV head's query rows / 256 of an attention) a call is refused
 * (RC_ERR_UNSUPPORTED).  Metadata out of these bounds (or a page id that
 * is not one of the pool's) is found on the device: the sequence is left out, such
 * a page is not written, and where it would be read page 0 is; nothing is read or
 * written out of bounds, and rc_paged_status reports RC_ERR_ARG; that call's
 * results are not valid.
 *
 * workspace: device memory of RC_PAGED_WORKSPACE_BYTES, 256-byte aligned,
 * zeroed once by the caller before its first use.  It holds the status word
 * and the partial results of split calls; each call leaves it ready for the
 * next.  Calls that share a workspace (captured graphs included) must not run
 * at the same time: issue them on one stream, or give each stream its own.
 * Every call only launches kernels on `stream`, on the device that is current
 * (which must be the stream's and the pointers'), and can be captured into a
 * graph once it has been called directly, and a graph replayed any number of
 * times.
 */
#define RC_PAGED_WORKSPACE_BYTES ((size_t)64 << 20)

typedef struct rc_paged_view {
    uint8_t *kcodes;
    uint8_t *vcodes;
    uint8_t *kscale;
    uint8_t *vscale;
    void *workspace;
    int pages;       /* >= 1 */
    int kv_heads;    /* 1 .. 1024 */
    int head_dim;    /* 64 or 128 */
    int page_tokens; /* 16, 32, 64 or 128 */
} rc_paged_view;

typedef struct rc_paged_batch {
    const int32_t *page_table;
    const int32_t *kv_len;
    const int32_t *q_start; /* not read by rc_paged_evict */
    int seqs;               /* 1 .. 65535 */
    int table_pages;        /* row length of page_table */
    int tokens;             /* rows of K, V, Q, out (>= 0) */
    int max_new;            /* >= 0 */
    int max_kv;             /* 0 .. table_pages * page_tokens, at most 2^24 */
} rc_paged_batch;

/*
 * Write each sequence's new tokens into its pages: K turned at the tokens'
 * positions (as rc_rope_axes, unrounded), K and V quantised as above.  K, V:
 * device bf16 [tokens][kv_heads][head_dim], tokens k_stride / v_stride elements
 * apart; positions: device int32 [axes][tokens], axes pos_stride apart.  The
 * pages must already be in page_table.  Two sequences must not write to one page.
 * A sequence whose n is larger than its kv_len is left out (RC_ERR_ARG later).
 */
int rc_paged_write(const rc_paged_view *view, const rc_paged_batch *batch, const void *K_bf16, int64_t k_stride,
                   const void *V_bf16, int64_t v_stride, const int32_t *positions, int64_t pos_stride,
                   const rc_rope_plan *plan, void *stream);

/*
 * out = softmax(q . k / sqrt(head_dim)) v over the sequence's cached tokens, for
 * each of its new tokens and each of `heads` query heads; query head g reads
 * KV head g / (heads / kv_heads).  With causal != 0 new token i sees tokens
 * 0 .. kv_len - n + i, else all kv_len.  Q is bf16, already turned
 * (rc_rope_axes), [tokens][heads][head_dim]; out is bf16 of the same layout;
 * lse (may be NULL) is fp32 [tokens][heads], the natural logarithm of the sum
 * of exp(scores).  A query that sees nothing gets zeros and lse = -infinity.
 * heads must be a multiple of kv_heads; out must share no element with Q (RC_ERR_ARG).
 * Up to 16 rows per KV head, here and in rc_paged_accumulate, a row of Q is held in
 * fp16 relative to its largest value: what lies under 2^-32 of that loses bits.
 */
int rc_paged_attend(const rc_paged_view *view, const rc_paged_batch *batch, const void *Q_bf16, int64_t q_stride,
                    int heads, void *out_bf16, int64_t out_stride, float *lse, int causal, void *stream);

/*
 * The attention weight that each cached token received from the new tokens'
 * queries: out[s][h][j] = scores[s][h][j] + sum over the queries of KV head h
 * that see token j of exp(q . k_j / sqrt(head_dim) - lse).  lse as
 * rc_paged_attend gives it; a row whose lse is -infinity adds nothing.
 * scores, out: device fp32 [seqs][kv_heads][score_stride], score_stride >=
 * max_kv; out may be scores, other overlaps are refused (RC_ERR_ARG).  Entries kv_len .. max_kv - 1 are copied
 * unchanged, entries past max_kv not touched.  Every entry is summed in one fixed order: the
 * same inputs give the same bits.
 */
int rc_paged_accumulate(const rc_paged_view *view, const rc_paged_batch *batch, const void *Q_bf16, int64_t q_stride,
                        int heads, const float *lse, const float *scores, float *out, int64_t score_stride,
                        int causal, void *stream);

/*
 * Cut each sequence, per KV head, to at most `keep` tokens: its last `recent`
 * tokens and, of the others, those with the largest scores (equal scores: the
 * lower index first; -0 equals +0; a NaN counts as the largest).  The kept tokens' codes and scales
 * are copied, in order, to the pages of dst_table [seqs][dst_pages] (token i of
 * the result in page i / P, place i % P); a sequence of at most `keep` tokens
 * is copied whole.  The source pages are only read, so they may be shared;
 * no destination page may be a source page or appear twice.
 *   kept [seqs][kv_heads][keep]: the kept tokens' old indices, ascending; -1 past the end
 *   kv_len_out [seqs]: min(kv_len, keep); may be the batch's kv_len
 *   scores_out (may be NULL) [seqs][kv_heads][keep]: the kept tokens' scores; 0 past the end;
 *       must not overlap scores (RC_ERR_ARG)
 * Errors: RC_ERR_ARG also for keep < 1, recent outside 0 .. keep, or
 * min(keep, max_kv) tokens that do not fit dst_pages pages.
 */
int rc_paged_evict(const rc_paged_view *view, const rc_paged_batch *batch, const float *scores, int64_t score_stride,
                   int keep, int recent, const int32_t *dst_table, int dst_pages, int32_t *kept, int32_t *kv_len_out,
                   float *scores_out, void *stream);

/* Synchronise `stream` and report what the calls on this workspace found:
   RC_OK, RC_ERR_ARG (bad metadata, see above), RC_ERR_TIMEOUT (a kernel gave
   up a bounded wait) or RC_ERR_CUDA.  The status word is cleared. */
int rc_paged_status(const rc_paged_view *view, void *stream);

/* Test support: the longest one wait of a later paged call may take, in ns
   (default 2 s; process-wide; as rc_cache_set_wait_limit). */
int rc_paged_set_wait_limit(uint64_t ns);

/* ---- the paged cache in 4 bits ------------------------------------------------ */
/*
 * The paged cache above at 4.5 bits a value: E2M1 codes (0, 0.5, 1, 1.5, 2, 3, 4,
 * 6 and their negatives) with a scale byte per token, head and 16 dims.  Pages (P =
 * page_tokens: 16, 32, 64 or 128), device memory, 16-byte aligned:
 *   kcodes [pages][kv_heads][P][head_dim / 2]  dims 2i (low bits) and 2i + 1 of a token
 *   vcodes [pages][kv_heads][head_dim][P / 2]  tokens 2i (low bits) and 2i + 1 of a dim
 *   kscale, vscale [pages][kv_heads][head_dim / 16][P]
 * A scale byte has 5 bits of exponent and 3 of fraction, without a sign: byte b
 * stands for the fp16 number with the bits b << 7 (2^-17 to 2^-14 in steps of 2^-17,
 * then eighths of each power of two).  A block's scale s is the least with max |x| <=
 * 6 s, at most 10,240 (byte 226), so magnitudes over 61,440 saturate; a code is the
 * one nearest to x / s (ties to the code with an even number), of the exact turn for K (whose
 * zeros may have either sign).
 * Blocks of zeros have scale 0.  Every value is then an exact fp16 and bf16 number.
 * All scale bytes of a row (a token's K or V of a head) that holds an infinity or a
 * NaN are 255, its codes 0, and it reads as NaN.  Scale bytes 227 .. 254, and 255 in a part
 * of a row, are not produced; tokens that have them read as some number, infinity or NaN.
 *
 * Metadata (rc_paged_batch), workspace, streams, graphs and what happens to
 * metadata out of bounds are as for the paged cache; a workspace can serve both
 * kinds of cache under the same rule.
 */
typedef struct rc_paged4_view {
    uint8_t *kcodes;
    uint8_t *vcodes;
    uint8_t *kscale;
    uint8_t *vscale;
    void *workspace; /* RC_PAGED_WORKSPACE_BYTES, as in rc_paged_view */
    int pages;       /* >= 1 */
    int kv_heads;    /* 1 .. 1024 */
    int head_dim;    /* 64 or 128 */
    int page_tokens; /* 16, 32, 64 or 128 */
} rc_paged4_view;

/*
 * Write each sequence's new tokens into its pages: K turned at the tokens'
 * positions (as rc_rope_turn, unrounded), K and V quantised as above.  Arguments and errors as
 * rc_paged_write, with a form of the cache's head_dim; form NULL: K is stored as it comes, and
 * positions are not read (may be NULL).  A page that gets new tokens belongs to one sequence
 * and stands once in the part of its row that is written: V's words hold 16 tokens and
 * are written whole, older tokens with the bits that they have.
 */
int rc_paged4_write(const rc_paged4_view *view, const rc_paged_batch *batch, const void *K_bf16, int64_t k_stride,
                    const void *V_bf16, int64_t v_stride, const int32_t *positions, int64_t pos_stride,
                    const rc_rope_form *form, void *stream);

/*
 * Attention of each sequence's new tokens over its pages; arguments and errors
 * as rc_paged_attend.  A row of Q is held in fp16 relative to its largest value: what lies under
 * 2^-32 of that loses bits.  Scores are fp32: a row with one of 2^126 or more in magnitude reads as some
 * number, infinity or NaN.
 */
int rc_paged4_attend(const rc_paged4_view *view, const rc_paged_batch *batch, const void *Q_bf16, int64_t q_stride,
                     int heads, void *out_bf16, int64_t out_stride, float *lse, int causal, void *stream);

/* As rc_paged_status, for the calls on this view's workspace. */
int rc_paged4_status(const rc_paged4_view *view, void *stream);

/* Number of occupied slots of `layer`, or a negative status. */
int rc_cache_occupancy(const rc_cache *h, int layer);

/* Sum of all deltas applied so far. */
int64_t rc_cache_delta_total(const rc_cache *h);

/* Number of kernel launches this handle has made (for launch accounting). */
int64_t rc_cache_launch_count(const rc_cache *h);

/*
 * How the attention call treats the KV tiles of one ring (host only: no
 * device, no handle).  grp[0 .. slots) is the ring's write group per slot
 * (-1 = empty); tile t covers slots [128 t, min(128 t + 128, slots)).
 *   uniform[t / 64] bit t % 64: every slot of tile t holds the same write
 *     group, so one K and one V scale per head cover it (the fast path);
 *   split[t] = b in 1..127: tile t has 128 slots, [128 t, 128 t + b) hold one
 *     write group and [128 t + b, 128 t + 128) another (where a write's run of
 *     slots ends inside the tile; the two-run path); otherwise 0.
 * Every other tile takes the general path (per-slot scales and validity).
 * uniform (4 words) and split (256 bytes) are caller-owned host memory.
 * Errors: RC_ERR_ARG if a pointer is NULL or slots is outside 1 .. 32768.
 */
int rc_tile_kinds(const int32_t *grp, int slots, uint64_t *uniform, uint8_t *split);

#ifdef __cplusplus
}
#endif

#endif /* RC_H */
