/*
 * ltx3drope.h - fused 3D rotary position embedding (RoPE) of the LTX-2.5
 * diffusion video decoder, for AMD Instinct MI355X (gfx950).
 *
 * The operation is the one described on the sglang PR #35698 page
 * ("fused LTX-2.5 decoder 3D RoPE", prhub.com.cn): sections "Implementation
 * breakdown" (steps 1-4) and "Key source snippets" (the JIT wrapper and the
 * CUDA kernel).  Every decoder attention block rotates its Q and K over the
 * latent (T, H, W) token grid with per-axis cos/sin tables that all blocks
 * on one grid share.
 *
 * Tensor layout (all four tensors): contiguous [B, T, H, W, heads, head_dim]
 * of one dtype; token n = (t*H + h)*W + w inside each batch element.  The
 * head dimension is cut into a t chunk of dim_t channels, an h chunk of
 * dim_h channels and a w chunk of dim_w channels, in that order
 * (head_dim == dim_t + dim_h + dim_w, each even and > 0).  Inside a chunk the
 * channels form interleaved pairs (x[2j], x[2j+1]).
 *
 * Tables: for an axis of length L and width d, entry (p, i), p in [0, L),
 * i in [0, d/2), holds cos and sin of p * base^(-2i/d), evaluated in float64
 * on the host and rounded once to fp32.  (The page names the builder but not
 * its formula; this is the textbook inverse-frequency reading with integer,
 * tile-local positions, since the cache key has no offset.)
 *
 * Rotation of one pair (e, o) with (c, s) from the token's table row, every
 * operation an fp32 IEEE round-to-nearest-even step and no fused
 * multiply-add ("Key source snippets", the kernel's pair-rotation helper):
 *     e' = (e*c) - (o*s),   o' = (e*s) + (o*c)
 * then cast back to the tensor dtype (bf16: round to nearest, ties to even;
 * fp32: identity).  Q and K use the same (c, s).  ltx3drope_apply_qk writes
 * out of place and never modifies its inputs; the shard entry point can also
 * rotate in place (see ltx3drope_shard_t).
 *
 * All functions are thread-safe, never throw, and return a status code
 * (LTX3DROPE_OK == 0, negative on error) unless stated otherwise.  Pointers
 * named q, k, q_out, k_out are device pointers owned by the caller.  Table
 * handles are owned by the library and reference counted.  A "stream" is a
 * hipStream_t passed as void* (NULL = the device's null stream).
 *
 * Beside it stand the operations around the rotation: a shard of the grid,
 * the rotate-half form, patchify, the DiT frequency grid, and the rest of a
 * transformer block: norms before and after it with gate, scaled residual and
 * the next modulated norm, the gated feed-forward block, and the linear layer
 * in 8-bit integers.  Each is documented at its declaration.
 */
#ifndef LTX3DROPE_H
#define LTX3DROPE_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define LTX3DROPE_VERSION 1

/* ---- status codes ------------------------------------------------------ */
enum {
    LTX3DROPE_OK = 0,
    LTX3DROPE_E_INVALID = -1,        /* an argument is malformed (null handle, bad size, bad base) */
    LTX3DROPE_E_UNSUPPORTED = -2,    /* the precheck rejects the tensors; nothing was launched */
    LTX3DROPE_E_TABLE_MISMATCH = -3, /* the tables do not belong to this grid / split / device */
    LTX3DROPE_E_HIP = -4,            /* a HIP runtime call failed */
    LTX3DROPE_E_NOMEM = -5           /* a host or device allocation failed */
};

/* ---- element types ----------------------------------------------------- */
enum { LTX3DROPE_DTYPE_F32 = 0, LTX3DROPE_DTYPE_BF16 = 1 };

/* ---- precheck reason codes (ltx3drope_can_use) ------------------------- */
enum {
    LTX3DROPE_REASON_OK = 0,
    LTX3DROPE_REASON_NULLPTR = 1,        /* a tensor pointer or the table handle is NULL */
    LTX3DROPE_REASON_DTYPE = 2,          /* dtype is neither F32 nor BF16 */
    LTX3DROPE_REASON_NONPOSITIVE_DIM = 3,/* B, T, H, W, heads or head_dim <= 0 */
    LTX3DROPE_REASON_SPLIT_ODD = 4,      /* a table chunk width is odd or <= 0 (tables carry the split) */
    LTX3DROPE_REASON_SPLIT_SUM = 5,      /* head_dim != dim_t + dim_h + dim_w */
    LTX3DROPE_REASON_TABLE_GRID = 6,     /* the tables were built for another (T, H, W) */
    LTX3DROPE_REASON_TABLE_DEVICE = 7,   /* the tables live on another device than the tensors */
    LTX3DROPE_REASON_ALIGN = 8,          /* a pointer is not aligned to one pair (2 elements) */
    LTX3DROPE_REASON_OVERLAP = 9,        /* an output overlaps an input or the other output */
    LTX3DROPE_REASON_TOO_LARGE = 10,     /* a batch element of 2^32 elements or more, a size of 2^31 or more,
                                            or more than 2^48 elements in all */
    LTX3DROPE_REASON_NOT_DEVICE_PTR = 11,/* a pointer is not device memory of the tables' device */
    LTX3DROPE_REASON_HOST_MODE = 12,     /* host-table test mode: apply calls refused, nothing launched (a name
                                            for that refusal; the precheck itself never returns it) */
    LTX3DROPE_REASON_EXTENT = 13         /* a pointer's device allocation ends before the tensor does */
};

/* ---- options (ltx3drope_set_option / ltx3drope_get_option) ------------- */
enum {
    LTX3DROPE_OPT_PATH = 1,        /* 0 auto (gate decides), 1 force fast kernel, 2 force plain kernel */
    LTX3DROPE_OPT_GATE = 2,        /* 0 off (trust fast), 1 verify the first call per key (default), 2 verify every call */
    LTX3DROPE_OPT_FORCE_GATE_MISMATCH = 3, /* 1: every verification reports a mismatch (tests the fallback) */
    LTX3DROPE_OPT_HOST_TABLES = 4, /* 1: tables are built in host memory and nothing touches HIP (CPU tests of the
                                      cache and the precheck); can_use still reports the precheck's verdict
                                      (memory checks skipped), and every apply call with such tables returns
                                      E_UNSUPPORTED without launching */
    LTX3DROPE_OPT_LOG = 5          /* 1: one stderr line per gate decision */
};

/* ---- gate states (ltx3drope_gate_state) -------------------------------- */
enum { LTX3DROPE_GATE_UNSEEN = 0, LTX3DROPE_GATE_TRUSTED = 1, LTX3DROPE_GATE_DISABLED = 2 };

typedef struct ltx3drope_tables* ltx3drope_tables_t;

typedef struct {
    int device;
    int64_t T, H, W;
    int64_t dim_t, dim_h, dim_w;
    double base;
    /* device (or, in host-table mode, host) address of the packed tables: float pairs (cos, sin),
       t section [T][dim_t/2], then h section [H][dim_h/2], then w section [W][dim_w/2] */
    const void* packed;
    int64_t packed_pairs;
} ltx3drope_tables_desc;

typedef struct {
    int64_t cache_hits, cache_misses, cache_evictions, cache_live;
    int64_t tables_alive;               /* table objects not yet freed (cache- or caller-held) */
    int64_t gate_verifications, gate_trusted, gate_disabled;
    int64_t fast_launches, plain_launches;
    int64_t rejected;                   /* apply_qk calls refused by the precheck */
} ltx3drope_stats_t;

/*
 * ltx3drope_tables_build - find or build the per-axis tables of one grid.
 *
 * The page's cached table lookup ("Implementation breakdown", step 1): the key
 * is (device, T, H, W, dim_t, dim_h, dim_w, base); a hit returns the cached
 * tables; a miss builds them (float64 on the host, rounded once to fp32),
 * uploads them with hipMemcpyAsync on `stream` followed by a synchronization of
 * that stream, and inserts them.  The cache holds at most 16 entries and
 * evicts first-in first-out (a hit does not refresh an entry).
 *
 * On success *out receives a handle holding one reference for the caller;
 * release it with ltx3drope_tables_release.  Eviction only drops the cache's
 * own reference, so a handle held by a caller stays valid after eviction.
 * Errors: E_INVALID (null out, T/H/W <= 0, a dim odd or <= 0, base not finite
 * or <= 0, device < 0), E_NOMEM, E_HIP.
 */
int ltx3drope_tables_build(int device, int64_t T, int64_t H, int64_t W,
                           int64_t dim_t, int64_t dim_h, int64_t dim_w, double base,
                           void* stream, ltx3drope_tables_t* out);

/* Drop one reference; the table memory is freed when the last one goes (hipFree waits for the
   device's outstanding work).  E_INVALID on NULL. */
int ltx3drope_tables_release(ltx3drope_tables_t tables);

/* Describe a table set (grid, split, base, device, packed address).  E_INVALID on NULL arguments. */
int ltx3drope_tables_describe(ltx3drope_tables_t tables, ltx3drope_tables_desc* out);

/* Copy the six tables to caller-owned host arrays of fp32, row-major [L][d/2] each (any pointer may
   be NULL to skip it).  Synchronous (device-wide copy).  E_INVALID, E_HIP. */
int ltx3drope_tables_read(ltx3drope_tables_t tables, float* cos_t, float* sin_t, float* cos_h,
                          float* sin_h, float* cos_w, float* sin_w);

/* Drop the cache's references to every entry (tables still held by callers stay valid). */
int ltx3drope_cache_clear(void);

/*
 * ltx3drope_can_use - the precheck ("Key source snippets", the JIT wrapper's
 * can_use predicate, plus rules of this library).
 *
 * Returns 1 if ltx3drope_apply_qk would launch for these arguments, 0 if it
 * would refuse.  q_out and k_out may both be NULL: then only the inputs are
 * checked (for a caller that allocates fresh outputs afterwards).  When
 * `reason` is not NULL it receives an LTX3DROPE_REASON_* code (the first
 * failing rule in the order of the enum).  Rules: no NULL
 * pointer or handle; dtype F32 or BF16; B, T, H, W, heads, head_dim > 0;
 * table split widths even and > 0 and summing to head_dim; tables built for
 * (T, H, W); every pointer aligned to one pair (8 B for F32, 4 B for BF16);
 * neither output overlapping an input or the other output; each size below
 * 2^31, fewer than 2^32 elements per batch element (8 GiB of bf16, 16 GiB of
 * fp32) and at most 2^48 in all (a tensor of 2^32 elements or more runs as
 * several launches of whole batch elements); all four pointers
 * device memory of the tables'
 * device, each inside an allocation large enough for the whole tensor
 * (checked last, REASON_NOT_DEVICE_PTR then REASON_EXTENT; skipped in
 * host-table mode).  Pure host logic: no launch, no allocation, no synchronization
 * (pointer attributes are queried from the HIP runtime).
 */
int ltx3drope_can_use(const void* q_out, const void* k_out, const void* q, const void* k, int dtype,
                      int64_t B, int64_t T, int64_t H, int64_t W, int64_t heads, int64_t head_dim,
                      ltx3drope_tables_t tables, int* reason);

/*
 * ltx3drope_apply_qk - rotate Q and K in one launch ("Key source snippets":
 * the wrapper writes fresh q_out and k_out with one kernel launch).
 *
 * q, k: inputs [B, T, H, W, heads, head_dim]; q_out, k_out: caller-allocated
 * outputs of the same shape and dtype (the caller allocates them fresh; they
 * must not overlap the inputs).  The precheck runs first; on failure nothing
 * is launched and E_UNSUPPORTED (or E_TABLE_MISMATCH for REASON_TABLE_GRID /
 * REASON_TABLE_DEVICE) is returned.  Otherwise the work is enqueued on
 * `stream` and the call returns without waiting, except on the first call of
 * a configuration while the bit-exact gate is on: then the fast kernel's
 * output is checked bit for bit against the plain kernel on the device and
 * the stream is synchronized once ("Implementation breakdown", step 4: first
 * call verified; equal -> the fast path is trusted, unequal -> permanent
 * fallback to the plain path for that configuration).  The gate's
 * configuration key is (device, dtype, B, T, H, W, heads, head_dim, dim_t,
 * dim_h, dim_w, the tables' T, H, W and the shard offsets): each shard
 * placement is verified on its own first call.  The comparison is of raw bits: both kernels write a NaN
 * result as the canonical quiet NaN (0x7FC00000 fp32, 0x7FC0 bf16).  On a
 * stream under graph capture an unverified configuration runs the plain
 * kernel and stays unverified (the check cannot wait for its count there).
 * The first verification on a device allocates that device's 256-byte
 * counter, kept until the process ends: E_NOMEM if the device is out of
 * memory, E_HIP for any other failed HIP call or launch.
 */
int ltx3drope_apply_qk(void* q_out, void* k_out, const void* q, const void* k, int dtype,
                       int64_t B, int64_t T, int64_t H, int64_t W, int64_t heads, int64_t head_dim,
                       ltx3drope_tables_t tables, void* stream);

/*
 * ltx3drope_apply_qk_noalloc - ltx3drope_apply_qk for callers that cannot allocate device
 * memory: code under HIP graph capture, tight serving loops, harnesses that forbid hipMalloc.
 * Same arguments, precheck, kernels, gate and results as ltx3drope_apply_qk (the caller passes
 * the inputs and the outputs), but it calls no hipMalloc, hipFree or other allocating routine:
 * the gate's verification counts its mismatches in a static 256-byte device array of the
 * library (one copy per GPU, held until the process ends) instead of the counter block
 * ltx3drope_apply_qk allocates on a device's first verification.  The counter is cleared by a
 * kernel before each use; its size does not depend on the input, so every input the precheck
 * accepts fits.  Every call on one GPU shares that array,
 * which keeps the last call's contents: verifications on one GPU are serialized by a host mutex
 * of the library from the counter's clearing to its read-back, and calls that overlap on one GPU
 * without it (from outside the library) would race.  The tables come from
 * ltx3drope_tables_build beforehand (which does allocate, once per grid).  E_UNSUPPORTED also for
 * tables of device index 64 or above.
 */
int ltx3drope_apply_qk_noalloc(void* q_out, void* k_out, const void* q, const void* k, int dtype,
                               int64_t B, int64_t T, int64_t H, int64_t W, int64_t heads, int64_t head_dim,
                               ltx3drope_tables_t tables, void* stream);

/*
 * Shards.  A sequence- or tile-parallel rank holds a slab of a larger token
 * grid; its tokens must take the table rows of their global coordinates.
 * (Positions on the page are tile-local because the table cache key carries
 * no offset: "Implementation breakdown", step 1.  The descriptor below is the
 * offset that splitting one grid over several devices needs.)
 *
 * t_offset, h_offset, w_offset: global frame / row / column of the tensor's
 * first frame / row / column.  The tables passed with a shard describe the
 * whole grid: for each axis offset + local size <= the tables' size, else
 * REASON_TABLE_GRID.  A token at local (t, h, w) is rotated with table rows
 * (t + t_offset, h + h_offset, w + w_offset).
 * inplace: 1 allows q_out == q and k_out == k exactly (partial overlaps stay
 * refused).  In-place calls cannot be checked by the bit-exact gate (the
 * inputs are overwritten); they use the fast kernel only once the
 * configuration is TRUSTED (or the gate is off, or the fast path is forced),
 * and the plain kernel otherwise.  A NULL descriptor means zero offsets,
 * out of place.
 */
typedef struct {
    int64_t t_offset, h_offset, w_offset;
    int32_t inplace;
    int32_t reserved;  /* must be 0 */
} ltx3drope_shard_t;

/* The precheck of a shard call: as ltx3drope_can_use, with the grid rule replaced by the shard's
   containment rule and the in-place exception to the overlap rule.  A malformed descriptor (a
   negative offset, an inplace value other than 0 or 1, or a non-zero reserved field) fails with
   REASON_TABLE_GRID before any other rule is looked at. */
int ltx3drope_can_use_shard(const void* q_out, const void* k_out, const void* q, const void* k, int dtype,
                            int64_t B, int64_t T, int64_t H, int64_t W, int64_t heads, int64_t head_dim,
                            const ltx3drope_shard_t* shard, ltx3drope_tables_t tables, int* reason);

/* ltx3drope_apply_qk on a shard of the tables' grid (see above); B, T, H, W are the tensor's local
   sizes.  Same statuses as ltx3drope_apply_qk; the gate key is the same as for an unsharded call of
   the same local shape (offsets do not change which code runs). */
int ltx3drope_apply_qk_shard(void* q_out, void* k_out, const void* q, const void* k, int dtype,
                             int64_t B, int64_t T, int64_t H, int64_t W, int64_t heads, int64_t head_dim,
                             const ltx3drope_shard_t* shard, ltx3drope_tables_t tables, void* stream);

/*
 * Rotate-half ("NeoX") RoPE with a position-gathered cos/sin cache: the text
 * encoder's rotary (sglang PR #24660 page, "Key source snippets", the Gemma3
 * rotary application; "Implementation breakdown", step 2).
 *
 * q [tokens, q_heads, head_dim], k [tokens, k_heads, head_dim] (the head
 * counts may differ), contiguous, dtype F32 or BF16; positions [tokens] int64
 * device array; cache [max_position, head_dim] of cache_dtype (F32 or BF16)
 * holding cos in columns [0, head_dim/2) and sin in [head_dim/2, head_dim).
 * For i < head_dim/2 with (c, s) = the token's cache row at i, converted to
 * q's dtype:
 *     out[i]            = R( R(x[i] * c)            + R(-x[i + head_dim/2] * s) )
 *     out[i + head_dim/2] = R( R(x[i + head_dim/2] * c) + R(x[i] * s) )
 * where R rounds an fp32 result to q's dtype (bf16: nearest even).  The
 * outputs may alias their own input exactly (q_out == q, k_out == k); every
 * other overlap is refused.  A position outside [0, max_position) is never
 * read: that token's outputs are set to NaN and counted (see
 * ltx3drope_neox_position_errors).  One launch for Q and K, on `stream`.
 * Reasons: NULLPTR, DTYPE (q or cache dtype), NONPOSITIVE_DIM, SPLIT_ODD
 * (odd head_dim), ALIGN (element alignment; positions 8 B), OVERLAP,
 * TOO_LARGE (a tensor or the cache of 2^32 elements or more, or a size of
 * 2^31 or more), NOT_DEVICE_PTR,
 * TABLE_DEVICE (pointers on different devices), EXTENT.  can_use accepts
 * q_out and k_out both NULL (fresh outputs: only the inputs are checked);
 * apply_qk needs both.  tokens = 0 is an empty call: the other sizes and the
 * dtypes are checked, no pointer is looked at (an empty tensor's may be NULL),
 * can_use returns 1 and apply_qk returns OK without launching.  The rules are
 * checked in this order and the first that fails names the reason: with
 * tokens = 0, DTYPE, NONPOSITIVE_DIM (q_heads, k_heads, head_dim or
 * max_position <= 0), SPLIT_ODD, TOO_LARGE (a size of 2^31 or more, or a cache
 * of 2^32 elements or more); otherwise NULLPTR, DTYPE, NONPOSITIVE_DIM,
 * SPLIT_ODD, ALIGN (q_out, k_out, q, k to their element size, the cache to
 * its own, positions to 8 B), TOO_LARGE, OVERLAP (an output over an input
 * other than its own exactly, over the other output, the positions or the
 * cache), then the device-memory rules.  apply_qk returns
 * E_UNSUPPORTED for any of these; the first call on a device allocates the
 * device's 256-byte counter (E_NOMEM when out of memory, E_HIP for another
 * HIP failure), and a failed launch gives E_HIP.
 */
int ltx3drope_neox_can_use(const void* q_out, const void* k_out, const void* q, const void* k, int dtype,
                           int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t head_dim,
                           const int64_t* positions, const void* cache, int cache_dtype, int64_t max_position,
                           int* reason);
int ltx3drope_neox_apply_qk(void* q_out, void* k_out, const void* q, const void* k, int dtype,
                            int64_t tokens, int64_t q_heads, int64_t k_heads, int64_t head_dim,
                            const int64_t* positions, const void* cache, int cache_dtype, int64_t max_position,
                            void* stream);
/* Number of (token, tensor) pairs whose position was outside the cache since the last reset, on
   `device`.  Synchronizes the device.  reset = 1 clears the count afterwards. */
int ltx3drope_neox_position_errors(int device, int reset, int64_t* count);

/*
 * Stage-5 space-to-depth of the diffusion decoder (sglang PR #34471 page,
 * "Key source snippets", _patchify) and its inverse (_unpatchify):
 *     x (B, C, F, H, W) <-> y (B, C*p*p, F, H/p, W/p)
 *     y[b, (c*p + pw)*p + ph, f, hh, ww] = x[b, c, f, hh*p + ph, ww*p + pw]
 * i.e. channels packed as (channel, width offset, height offset).  Both tensors
 * contiguous, elements of elem_bytes = 1, 2, 4 or 8 bytes (the op moves data
 * and never looks at values, so it is exact for every dtype).  B, C, F, H, W
 * are always the unpatched sizes.  A size of 0 is an empty call: OK, nothing
 * launched, no pointer looked at (an empty tensor's may be NULL).  E_INVALID:
 * a size < 0, p <= 0, H or W not a multiple of p, elem_bytes not 1/2/4/8,
 * NULL pointers of a non-empty call.  E_UNSUPPORTED: 2^32
 * elements or more (or C*p*p of 2^31 or more), pointers not aligned to one
 * element, overlapping tensors,
 * not device memory of one device, or allocations smaller than the tensors.
 * Asynchronous on `stream`.  E_NOMEM / E_HIP: the device's first call could not
 * allocate the library's 256-byte per-device counter block; E_HIP: a failed
 * launch.
 */
int ltx3drope_patchify(void* y, const void* x, int elem_bytes, int64_t B, int64_t C, int64_t F, int64_t H,
                       int64_t W, int64_t p, void* stream);
int ltx3drope_unpatchify(void* x, const void* y, int elem_bytes, int64_t B, int64_t C, int64_t F, int64_t H,
                         int64_t W, int64_t p, void* stream);

/*
 * LTX DiT RoPE frequency grid, generated on the device (sglang PR #24660 page,
 * "Key source snippets", the DiT's frequency generation; "Implementation
 * breakdown", step 2: generated on the target device in the requested
 * precision, keeping the official rounding trajectory):
 *     n = dim / num_rope_elems (integer division)
 *     out[i] = float32( theta ** linspace(0, 1, n)[i] * pi / 2 )
 * in float64 (double_precision = 1) or float32 (0), every step rounded to
 * nearest even in that precision: linspace as torch.linspace computes it (a
 * rounded step s = 1/(n-1); s*i for i < n/2, else 1 - s*(n-1-i) rounded once),
 * the correctly rounded power (theta first rounded to float32 in the float32
 * recipe), pi rounded to the working precision, an exact halving, and in the
 * float64 recipe one rounding to float32 at the end.
 * `out`: device memory of n floats (written by one kernel launch on `stream`,
 * asynchronous; its device is the current one).  *count (if not NULL) receives
 * n; n = 0 launches nothing and `out` may be NULL.
 * E_INVALID: theta not in [2^-126, FLT_MAX] (a normal float32), dim < 0,
 * num_rope_elems <= 0, n > 2^24, out NULL while n > 0.  E_UNSUPPORTED: `out`
 * is not device memory holding n floats.  E_HIP: the launch failed.
 */
int ltx3drope_dit_freq_grid(double theta, int64_t dim, int64_t num_rope_elems, int double_precision, float* out,
                            void* stream, int64_t* count);

/*
 * RMS norms before and after a transformer block, fused with the block's gate,
 * its scaled residual and the next norm's scale and shift.
 *
 * Row tensors are contiguous [batch, rows, dim] of `dtype` (F32 or BF16).
 * Vectors are contiguous and of `param_dtype` (F32, or BF16 with BF16 rows):
 * weights [dim]; gate, next_scale and next_shift [batch, dim].  Any vector may
 * be NULL; its factor is then 1 and its term 0.  With
 * hat(v) = v / sqrt(mean(v^2) + eps), per row of sample b and all in fp32:
 *     branch = (post_norm ? hat(y) : y) * (weight + weight_offset)
 *     r      = residual_scale * residual + gate_b * branch
 *     n      = hat(r) * (next_weight + weight_offset) * (1 + next_scale_b) + next_shift_b
 * each output rounded once to `dtype` (n is formed from the unrounded r).
 * weight_offset counts only where its weight is given.  mean(v^2) has to be
 * finite in fp32 (with an eps below 2^-110 the sum of the squares): a row whose
 * squares pass it gives zeros or NaN.
 *
 * after = 1: y, residual and r are required; next_norm = 1 also writes n.
 * after = 0 is the norm before a block alone: n from `residual`; y, weight,
 * gate and r must be NULL, post_norm 0, next_norm 1 and residual_scale 1.
 *
 * An output may be exactly one of the row inputs (r over residual, n over y);
 * every other overlap is refused.  batch = 0 or rows = 0 is an empty call: OK,
 * nothing launched, no pointer looked at.
 * E_INVALID: a NULL descriptor; eps not finite or <= 0; weight_offset or
 * residual_scale not finite; a flag other than 0 or 1 or a combination other
 * than the above.  E_UNSUPPORTED, with the reason in *reason (which may be
 * NULL), the first that fails of: DTYPE; NONPOSITIVE_DIM (dim <= 0, batch or
 * rows < 0); TOO_LARGE (dim > 16384, batch * rows of 2^31 or more, or batch >
 * 65535 where a [batch, dim] vector is given); NULLPTR; ALIGN (a pointer not
 * aligned to its element); OVERLAP; then NOT_DEVICE_PTR, TABLE_DEVICE (memory
 * of two devices) and EXTENT.  E_HIP: the launch failed.  Asynchronous on
 * `stream`; allocates nothing.
 */
typedef struct {
    int32_t dtype, param_dtype;
    int32_t after, post_norm, next_norm, reserved; /* reserved must be 0 */
    int64_t batch, rows, dim;
    float eps, weight_offset, residual_scale;
    const void *y, *residual, *weight, *gate, *next_weight, *next_scale, *next_shift;
    void *r, *n;
} ltx3drope_norm_t;
int ltx3drope_norm(const ltx3drope_norm_t* call, void* stream, int* reason);

/*
 * The gradients of ltx3drope_norm.  `r` is the forward's output r (after = 1)
 * or its input (after = 0); dr (may be NULL: zero) is the gradient that reaches
 * r past the next norm, dn (required with next_norm = 1, else NULL) that of n.
 * With v = dn * (next_weight + weight_offset) * (1 + next_scale_b):
 *     dR        = dr + (v - hat(r) * mean(v * hat(r))) / sqrt(mean(r^2) + eps)
 *     dresidual = residual_scale * dR
 *     q         = dR * gate_b * (weight + weight_offset)
 *     dy        = post_norm ? (q - hat(y) * mean(q * hat(y))) / sqrt(mean(y^2) + eps) : q
 * and the vectors' gradients, sums over rows (weights: over rows and samples)
 * held in fp32, in param_dtype.  dresidual is required, dy too with after = 1;
 * the vectors' gradients may each be NULL, and must be where the vector itself
 * is (dnext_shift alone needs no vector).  y may be NULL where nothing needs it
 * (no post norm, no gate and no weight); r where next_norm = 0.
 * `workspace`: ltx3drope_norm_backward_workspace bytes of device memory, 16-byte
 * aligned, that nothing else uses until the call's work on `stream` has run; 0
 * bytes where no vector's gradient is asked for (then it may be NULL).  Sums are
 * added in a fixed order: equal inputs give equal bits.  Empty calls write zeros
 * into the vectors' gradients.  Aliasing, statuses and reasons as above;
 * a workspace that is too small is E_INVALID.
 */
typedef struct {
    int32_t dtype, param_dtype;
    int32_t after, post_norm, next_norm, reserved;
    int64_t batch, rows, dim;
    float eps, weight_offset, residual_scale;
    const void *dr, *dn, *y, *r, *weight, *gate, *next_weight, *next_scale;
    void *dresidual, *dy, *dweight, *dgate, *dnext_weight, *dnext_scale, *dnext_shift;
    void* workspace;
    int64_t workspace_bytes;
} ltx3drope_norm_backward_t;
int ltx3drope_norm_backward(const ltx3drope_norm_backward_t* call, void* stream, int* reason);
/* Bytes of workspace for a call (its sizes and which gradients are not NULL; no pointer is looked
   at), or a negative status for a malformed descriptor. */
int64_t ltx3drope_norm_backward_workspace(const ltx3drope_norm_backward_t* call);

/*
 * The gated feed-forward block: both projections, the activation and the
 * product in one kernel.
 *     g = x Wg^T,  u = x Wu^T,  h = act(g) * u
 * x [tokens, dim], w_gate and w_up [hidden, dim], h [tokens, hidden], all
 * contiguous and of `dtype` (F32 or BF16); sums, activation and product in fp32,
 * h rounded once.  g and u (both or neither, [tokens, hidden] fp32 whatever the
 * dtype) receive the projections for the backward pass: in fp32, so that the
 * gradients carry no rounding of theirs.
 * `workspace`: ltx3drope_gated_ffn_workspace bytes of device memory, 16-byte
 * aligned, that nothing else uses until the call's work on `stream` has run.  It
 * is 0 (then workspace may be NULL) but where more than 16 tokens meet long sums
 * and few outputs: the sums are then split over the chip and their parts lie there.
 * tokens = 0 or hidden = 0 is an empty call: OK, nothing launched, no pointer
 * looked at.  E_INVALID: a NULL descriptor, an unknown activation, one of g and u without the other, a workspace that is too small.
 * E_UNSUPPORTED with the reason in *reason (which may be NULL), the first that
 * fails of: DTYPE; NONPOSITIVE_DIM (dim <= 0, tokens or hidden < 0); TOO_LARGE
 * (tokens, 2 * hidden or dim of 2^21 or more, or more than 2^23 output tiles of
 * 64 x 32: 2^34 outputs); NULLPTR; ALIGN (a pointer not
 * aligned to its element, the workspace not to 16 bytes); OVERLAP (an output or
 * the workspace over anything else); then NOT_DEVICE_PTR, TABLE_DEVICE (memory
 * of two devices) and EXTENT.  E_HIP: a launch failed.  Asynchronous on
 * `stream`; allocates nothing.
 */
enum { LTX3DROPE_ACT_SILU = 0, LTX3DROPE_ACT_GELU = 1, LTX3DROPE_ACT_GELU_TANH = 2 };
typedef struct {
    int32_t dtype, activation;
    int64_t tokens, dim, hidden;
    const void *x, *w_gate, *w_up;
    void* h;
    float *g, *u;
    void* workspace;
    int64_t workspace_bytes;
} ltx3drope_gated_ffn_t;
int ltx3drope_gated_ffn(const ltx3drope_gated_ffn_t* call, void* stream, int* reason);
/* Bytes of workspace for a call (its sizes, and the alignment of x and the weights), or a negative
   status for a malformed descriptor. */
int64_t ltx3drope_gated_ffn_workspace(const ltx3drope_gated_ffn_t* call);

/*
 * The gradients of ltx3drope_gated_ffn from the g and u that it kept:
 *     dg = dh * u * act'(g),  du = dh * act(g)
 *     dx = dg Wg + du Wu,  dw_gate = dg^T x,  dw_up = du^T x
 * dg and du are formed in fp32 and rounded once to `dtype` for the matrix cores;
 * the sums are held in fp32 and each output rounded once.  dx may be NULL, and
 * so may dw_gate and dw_up together; what is NULL is not computed.  Sums are
 * added in a fixed order: equal inputs give equal bits.  An empty call
 * (tokens = 0 or hidden = 0) writes zeros into what it is given.  Statuses and
 * reasons as above; every call that is not empty needs a workspace.
 */
typedef struct {
    int32_t dtype, activation;
    int64_t tokens, dim, hidden;
    const void *dh, *x, *w_gate, *w_up;
    const float *g, *u;
    void *dx, *dw_gate, *dw_up;
    void* workspace;
    int64_t workspace_bytes;
} ltx3drope_gated_ffn_backward_t;
int ltx3drope_gated_ffn_backward(const ltx3drope_gated_ffn_backward_t* call, void* stream, int* reason);
/* Bytes of workspace for a call (its sizes, the alignment of the operands, and which outputs are not
   NULL), or a negative status for a malformed descriptor. */
int64_t ltx3drope_gated_ffn_backward_workspace(const ltx3drope_gated_ffn_backward_t* call);

/*
 * Rows to 8-bit integers, one scale a row:
 *     scale[r] = max |x[r]| * (1/127),  q[r][c] = round(x[r][c] / scale[r])
 * in fp32, each step (and the constant) rounded once to nearest even, |q| <= 127.  x [rows, dim] of
 * `dtype` (F32 or BF16), q [rows, dim] int8, scale [rows] fp32, contiguous.  A
 * row of zeros gets scale 0 and zeros.  A row with a NaN or an infinity keeps
 * that as its scale and gets zeros: its products come out NaN.  rows = 0 is an
 * empty call.  E_UNSUPPORTED: DTYPE; NONPOSITIVE_DIM; TOO_LARGE (rows or dim of
 * 2^31 or more, or 2^48 elements or more); NULLPTR; ALIGN; OVERLAP;
 * NOT_DEVICE_PTR, TABLE_DEVICE, EXTENT.  E_HIP.  Asynchronous, allocates nothing.
 */
int ltx3drope_q8_quantize(int dtype, int64_t rows, int64_t dim, const void* x, void* q, float* scale, void* stream,
                          int* reason);

/*
 * A linear layer in 8-bit integers:
 *     y[m][n] = (sum_k a[m][k] * b[n][k]) * a_scale[m] * b_scale[n] + bias[n]
 * a [tokens, dim] and b [out, dim] int8, a_scale [tokens], b_scale and bias
 * [out] fp32 (bias may be NULL), y [tokens, out] of `dtype` (F32 or BF16),
 * contiguous.  The integer sums are exact; the rest is fp32, y rounded once.
 * `workspace` as for ltx3drope_gated_ffn.  tokens = 0 or out = 0 is an empty call.  E_INVALID: a NULL
 * descriptor, reserved not 0, a workspace that is too small.  E_UNSUPPORTED:
 * DTYPE; NONPOSITIVE_DIM; TOO_LARGE (dim > 131071, whose sums could pass 32
 * bits, tokens or out of 2^26 or more, or more than 2^23 output tiles of 64 x
 * 32); NULLPTR; ALIGN; OVERLAP;
 * NOT_DEVICE_PTR, TABLE_DEVICE, EXTENT.  E_HIP.  Asynchronous, allocates nothing.
 */
typedef struct {
    int32_t dtype, reserved;
    int64_t tokens, dim, out;
    const void *a, *b;
    const float *a_scale, *b_scale, *bias;
    void* y;
    void* workspace;
    int64_t workspace_bytes;
} ltx3drope_q8_matmul_t;
int ltx3drope_q8_matmul(const ltx3drope_q8_matmul_t* call, void* stream, int* reason);
int64_t ltx3drope_q8_matmul_workspace(const ltx3drope_q8_matmul_t* call);

/* Gate state of one unsharded configuration (tables built for the tensor's own grid, no offsets):
 * LTX3DROPE_GATE_*, or a negative status. */
int ltx3drope_gate_state(int device, int dtype, int64_t B, int64_t T, int64_t H, int64_t W,
                         int64_t heads, int64_t head_dim, int64_t dim_t, int64_t dim_h, int64_t dim_w);

/* Forget every gate decision (all configurations become UNSEEN). */
int ltx3drope_gate_reset(void);

int ltx3drope_set_option(int option, int64_t value);
int64_t ltx3drope_get_option(int option);

int ltx3drope_stats(ltx3drope_stats_t* out);
int ltx3drope_stats_reset(void);

/* Which kernel apply_qk would use for these arguments when the gate trusts the fast path:
   1 fast, 2 plain, or a negative status if the precheck fails (host rules only: device memory is
   not queried).  q_out and k_out may both be NULL: fresh outputs, which are 16-byte aligned. */
int ltx3drope_kernel_choice(const void* q_out, const void* k_out, const void* q, const void* k,
                            int dtype, int64_t B, int64_t T, int64_t H, int64_t W, int64_t heads,
                            int64_t head_dim, ltx3drope_tables_t tables);

/* Measurement helper: copy `bytes` (a multiple of 16, fewer than 2^32 - 64 vectors of 16 B, both
   pointers 16-B aligned, non-overlapping memory of one device) from src to dst with a plain streaming kernel
   on `stream` (the fast kernel's launch shape and cache hints, one read and one write stream); used
   as the bandwidth ceiling and to calibrate traffic counters.  E_INVALID on bad arguments, E_HIP. */
int ltx3drope_copy(void* dst, const void* src, int64_t bytes, void* stream);

const char* ltx3drope_status_string(int status);
const char* ltx3drope_reason_string(int reason);
int ltx3drope_version(void);

#ifdef __cplusplus
}
#endif

#endif /* LTX3DROPE_H */
