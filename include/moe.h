/*
 * moe.h -- C ABI of libmoe: the routed MXFP4 mixture-of-experts block of a
 * speculative-decode verify step, on one GB300 GPU (sm_103a), all experts
 * resident, no collectives.
 *
 * The block (pages cited by their vLLM module names):
 *   vllm.models.muse_spark.amd.mono.kernels.k3, stage list:
 *     A      the router's logits, in fp32
 *     route  the top 8 of every token (each CTA repeats the same routing);
 *            route_token starts from a sigmoid score (its summary is cut off)
 *     C, D   the local experts' gate_up and down projections, MXFP4 weights
 *     E      a norm of each pick's expert output, then the weighted sum
 *   vllm.models.muse_spark.amd.mono.kernels.k5, stage HA: fp32 router, top 8,
 *     ids and weights handed to the expert stage
 *   vllm.models.kimi_k3.amd.specialized_decode.mono.layer, k2_launch: the MoE
 *     arguments w_gate, bias, w13, w13s, w2, w2s and the output out [S, 7168].
 *
 * What is computed, for token t (0 <= t < S):
 *   L[t,e]   = sum_c x[t,c] * w_gate[e,c]  (fp32)  [+ logit_off[e]]
 *   s[t,e]   = sigmoid(L[t,e]);  sel = s + bias[e]
 *   picks    = the k experts with the largest sel (ties -> lower id),
 *              reported in ascending expert id; weight w_j = s_j / sum_j s_j
 *   g, u     = W1_e x_t, W3_e x_t   (W1 = rows 0..I-1 of w13, W3 = rows I..2I-1)
 *   h        = silu(g) * u;   y = W2_e h
 *   [post]   y <- y * rsqrt(mean(y^2) + norm_eps) * norm_w      (MOE_POST_NORM)
 *   out[t]   = sum_j w_j * y_j                                      (fp32)
 *
 * MXFP4 encoding (OCP Microscaling v1.0): an e2m1 element is a 4-bit code
 * (sign, 2 exponent bits with bias 1, 1 mantissa bit); an e8m0 scale byte b
 * means 2^(b-127) and covers 32 consecutive K-elements of one row.  Packed
 * rows are row-major with K contiguous: byte j holds element 2j in its low
 * nibble and element 2j+1 in its high nibble.  Scale bytes 0..254 (block
 * scales 2^-127 .. 2^127) are supported; the byte 255, NaN in the MX format,
 * latches MOE_ERR_BAD_SCALE on the device (the affected outputs are NaN).
 *
 * Precision: the expert GEMMs run on the tensor core's block-scaled e2m1 x
 * e4m3 path with fp32 accumulation.  The weights enter exactly; each bf16
 * token row enters as two e4m3 rows (leading and trailing 4 significant
 * bits) under a power-of-two scale per 32 elements, which is exact up to
 * 2^-17 of the block's largest magnitude; h = silu(g) * u enters the same
 * way from fp32 (about 9 significant bits, like a bf16 rounding).
 *
 * Conventions for every entry point:
 *   - All tensor pointers are DEVICE pointers (cudaMalloc'd or equivalent),
 *     16-byte aligned (the packed weights w13 and w2: 32-byte aligned),
 *     owned by the caller, and must stay valid until the
 *     work queued on `stream` has finished.  Nothing is allocated, freed or
 *     cached by the library on these paths; it keeps no state between calls
 *     except per-device kernel attributes.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *     stream).  Calls only enqueue work; they do not synchronise, except
 *     moe_device_status.  The library's kernels are launched with
 *     programmatic dependent launch: later kernels of a call read its inputs
 *     (weights, bias, x) before waiting on their predecessors, which is safe
 *     because the call's first kernel lets them start only once the stream's
 *     earlier work has completed.  A caller kernel launched the same way that
 *     writes an input must therefore not signal launch completion before the
 *     input is written.
 *   - `ws` is a device workspace of at least moe_workspace_bytes() bytes,
 *     256-byte aligned, prepared once with moe_workspace_init.  Its first
 *     bytes hold the device status word; calls that share one workspace must
 *     be ordered on one stream.
 *   - Return value: MOE_OK or a negative MOE_ERR_* code.  Host-side checks
 *     (arguments, shape, alignment, workspace size) run before anything is
 *     enqueued and enqueue nothing when they fail.  Errors found on the
 *     device (bad ids, bad scale bytes, a bounded wait that ran out) are
 *     latched in the workspace status word and reported by
 *     moe_device_status.  The library never aborts, traps or asserts.
 */
#ifndef MOE_H
#define MOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_ABI_VERSION 1

/* status codes */
#define MOE_OK                     0
#define MOE_ERR_INVALID_ARG       -1  /* NULL pointer, negative size, bad flags */
#define MOE_ERR_UNSUPPORTED_SHAPE -2  /* shape outside the supported set (below) */
#define MOE_ERR_ALIGNMENT         -3  /* a pointer is not 16-byte (w13, w2: 32; ws: 256) aligned */
#define MOE_ERR_WORKSPACE         -4  /* ws_bytes < moe_workspace_bytes() */
#define MOE_ERR_CUDA              -5  /* a CUDA runtime call or launch failed */
#define MOE_ERR_TIMEOUT           -6  /* device: a bounded wait ran out */
#define MOE_ERR_BAD_IDS           -7  /* device: an expert id outside [0, E) */
#define MOE_ERR_BAD_SCALE         -8  /* device: an e8m0 scale byte of 255 (NaN) */
#define MOE_ERR_NO_DEVICE         -9  /* current device is not sm_103 (GB300), or has too few SMs (moe_tree_attention) */
#define MOE_ERR_BAD_LENGTHS      -10  /* device: a request's length is negative or does not fit; a position past its table */
#define MOE_ERR_NO_PAGES         -11  /* device: the list of free pages is too short */
#define MOE_ERR_BAD_PARENT       -12  /* device: a drafted token's parent is not an earlier one */
#define MOE_ERR_BAD_PAGE         -13  /* device: a page id or slot outside the cache */

/* moe_shape.flags */
#define MOE_POST_NORM    1u  /* per-pick RMSNorm of y before the weighted sum */
#define MOE_LOGIT_OFFSET 2u  /* add logit_off[e] to the router logits */

/*
 * Problem shape.  Supported: S >= 1, S * k <= 1<<20; d % 128 == 0 and
 * 128 <= d <= 16384; I % 128 == 0 and 128 <= I <= 8192; 1 <= k <= 16;
 * k <= E <= 512; norm_eps >= 0 (used with MOE_POST_NORM only).
 */
typedef struct moe_shape {
    int32_t S;        /* token rows */
    int32_t d;        /* hidden size (K of gate_up, N-rows of down) */
    int32_t E;        /* experts */
    int32_t k;        /* picks per token */
    int32_t I;        /* expert intermediate size */
    uint32_t flags;   /* MOE_POST_NORM | MOE_LOGIT_OFFSET */
    float norm_eps;   /* RMSNorm epsilon */
} moe_shape;

/* ABI version of the loaded library (MOE_ABI_VERSION). */
int moe_abi_version(void);

/* Static English text for a status code; never NULL. */
const char* moe_strerror(int code);

/*
 * Workspace size for `shape` in *bytes.  Returns MOE_OK, MOE_ERR_INVALID_ARG
 * or MOE_ERR_UNSUPPORTED_SHAPE.  Pure host function.
 */
int moe_workspace_bytes(const moe_shape* shape, size_t* bytes);

/*
 * Clears the workspace's status block and its per-expert sort counters (the
 * first 6400 bytes, or ws_bytes if fewer; enqueued on `stream`).  Call once
 * after allocating a workspace, before its first use; the library's kernels
 * leave the counters cleared after every call that completes.
 */
int moe_workspace_init(void* ws, size_t ws_bytes, void* stream);

/*
 * Router + sigmoid top-k (k3 stages A and route; k5 HA).
 *   x         [S, d]  bf16, row-major
 *   w_gate    [E, d]  bf16, row-major (the router weight)
 *   bias      [E]     fp32, selection bias (affects the choice, not w_j)
 *   logit_off [E]     fp32, added to the logits when MOE_LOGIT_OFFSET is
 *                     set, else ignored (may be NULL)
 *   ids       [S, k]  int32 out: picks in ascending expert id
 *   weights   [S, k]  fp32 out: renormalised sigmoid of the picks, aligned
 *                     with ids
 */
int moe_route(const moe_shape* shape, const void* x, const void* w_gate,
              const float* bias, const float* logit_off,
              int32_t* ids, float* weights,
              void* ws, size_t ws_bytes, void* stream);

/*
 * Experts + combine (k3 stages C, D, E; k2_launch w13/w13s/w2/w2s/out).
 *   x         [S, d]        bf16
 *   ids       [S, k]        int32, expert of each pick, distinct within a
 *                           token, any order (an id outside [0, E), or one
 *                           repeated within its token, latches
 *                           MOE_ERR_BAD_IDS and that pick contributes
 *                           nothing)
 *   weights   [S, k]        fp32, aligned with ids
 *   w13       [E, 2I, d/2]  packed e2m1; rows 0..I-1 gate, I..2I-1 up
 *   w13s      [E, 2I, d/32] e8m0
 *   w2        [E, d, I/2]   packed e2m1
 *   w2s       [E, d, I/32]  e8m0
 *   norm_w    [d]           fp32 post-expert norm weight (MOE_POST_NORM),
 *                           else ignored (may be NULL)
 *   out       [S, d]        fp32, overwritten
 */
int moe_experts(const moe_shape* shape, const void* x,
                const int32_t* ids, const float* weights,
                const uint8_t* w13, const uint8_t* w13s,
                const uint8_t* w2, const uint8_t* w2s,
                const float* norm_w, float* out,
                void* ws, size_t ws_bytes, void* stream);

/*
 * The whole block: moe_route then moe_experts on one stream, with the same
 * arguments as those two (ids and weights are written, then consumed).
 */
int moe_forward(const moe_shape* shape, const void* x, const void* w_gate,
                const float* bias, const float* logit_off,
                const uint8_t* w13, const uint8_t* w13s,
                const uint8_t* w2, const uint8_t* w2s,
                const float* norm_w,
                int32_t* ids, float* weights, float* out,
                void* ws, size_t ws_bytes, void* stream);

/*
 * moe_forward with the step's input and outputs in HOST memory: x_host [S, d]
 * bf16 in, ids_host [S, k], weights_host [S, k], out_host [S, d] out, all
 * enqueued on `stream`.  An output in a small pinned buffer the GPU can
 * address (cudaHostAlloc'd or cudaHostRegister'ed memory; on GB300 over the
 * coherent CPU-GPU link), 16-byte aligned, is written in place by the kernels:
 * ids and weights when S <= 32 and S * k <= 128, out when S * d * 4 <= 256 KiB.
 * x is copied into the workspace, from a pinned buffer up to 1 MiB by a kernel
 * (which lets the router start meanwhile), else with one cudaMemcpyAsync; every
 * other host buffer (pageable, unaligned or larger) is staged through the
 * workspace with one cudaMemcpyAsync.  The weights (w_gate,
 * bias, logit_off, w13, w13s, w2, w2s, norm_w) stay device pointers.  The host
 * buffers must not be touched until the stream has been synchronised.
 * ids_host / weights_host may be NULL (then only out is returned).
 */
int moe_forward_host(const moe_shape* shape, const void* x_host, const void* w_gate,
                     const float* bias, const float* logit_off,
                     const uint8_t* w13, const uint8_t* w13s,
                     const uint8_t* w2, const uint8_t* w2s,
                     const float* norm_w,
                     int32_t* ids_host, float* weights_host, float* out_host,
                     void* ws, size_t ws_bytes, void* stream);

/*
 * moe_forward without a workspace argument, for callers that cannot allocate
 * device memory where they run the block (an operator or plugin interface
 * that passes only inputs and outputs, an application whose memory pool owns
 * the whole GPU, a serving loop that must not call cudaMalloc).  The pages have
 * no counterpart: their launchers always receive a scratch buffer.
 *
 * Scratch comes from a 32 MiB static device array inside the library, which
 * every GPU that uses this entry point holds until the process exits.  The
 * library's device modules load lazily (CUDA's default), so the 32 MiB are
 * reserved by the first call on a device, which loads the array's module and
 * looks up its device address once (cudaGetSymbolAddress, with that device
 * current).  Make that first call as a warm-up: before a memory pool claims
 * the whole GPU (else it fails with MOE_ERR_CUDA, reported on stderr) and
 * before any stream capture.  No call allocates or frees memory itself.
 * Shapes whose moe_workspace_bytes() exceeds 32 MiB are rejected with
 * MOE_ERR_WORKSPACE (S * k <= 256 at d = 4096, I = 1024, E = 256 fits), and
 * every argument check of moe_forward runs, with the same codes, before the
 * array is touched: a rejected call enqueues nothing.
 *
 * Every call on a device shares the one array, which keeps the previous
 * call's contents; each call clears its status block first.  Calls that
 * overlap on the GPU (other streams, other host threads) race on the array:
 * order them on one stream.  Arguments are those of moe_forward minus the
 * workspace; `status` (device int32[2], may be NULL) receives this call's
 * device status and detail (see moe_device_status) when the call's work is
 * done.
 */
int moe_forward_noalloc(const moe_shape* shape, const void* x, const void* w_gate,
                        const float* bias, const float* logit_off,
                        const uint8_t* w13, const uint8_t* w13s,
                        const uint8_t* w2, const uint8_t* w2s,
                        const float* norm_w,
                        int32_t* ids, float* weights, float* out,
                        int32_t* status, void* stream);

/*
 * The latent-MoE layer around the routed block, with a shared expert
 * (vllm.models.kimi_k3.amd.specialized_decode.mono.layer: K2b's stage list --
 * router parts and latent parts, route, the shared gate/up and its
 * activation, ug and down of the routed experts, the shared down, lnorm, up --
 * and k2_launch's arguments w_gate, bias, w_ld, w_sgu, w_sd, w13, w13s, w2,
 * w2s, ln_w, w_up, out [S, 7168]).  For token t:
 *   picks, w_j = the sigmoid top-k of x[t] (as moe_route, over H)
 *   xl        = x[t] . w_ld^T                   latent input, [LAT] (bf16)
 *   yl        = sum_j w_j * expert_j(xl)        the routed block at d = LAT
 *   zl        = yl * rsqrt(mean(yl^2) + norm_eps) * ln_w             (bf16)
 *   out[t]    = zl . w_up^T  +  (silu(g) * u) . w_sd^T,
 *               g, u = x[t] . w_sgu[0:SI]^T, x[t] . w_sgu[SI:2SI]^T  (fp32)
 * The pages give the stages and the argument names, not the formulas or the
 * formats: the dense weights carry no scale tensors and are bf16 here; the
 * latent norm is an RMSNorm with weight ln_w; the shared expert is a SwiGLU
 * expert on the layer input, its output added to the up projection's.  The
 * intermediate activations xl, zl and silu(g) * u are rounded to bf16, the
 * operand type of the dense products (bf16 x bf16 on the tensor cores, fp32
 * accumulation); every sum is fp32.
 *
 * Shape: H and LAT multiples of 128 (LAT <= 16384, H <= 16384), SI a
 * multiple of 128 or 0 (no shared expert), E, k, I as in moe_shape, S * k
 * <= 1<<20; flags may hold MOE_LOGIT_OFFSET only.
 */
typedef struct moe_latent_shape {
    int32_t S;        /* token rows */
    int32_t H;        /* hidden size of the layer input and output */
    int32_t LAT;      /* latent width: the routed experts' d */
    int32_t E;        /* routed experts */
    int32_t k;        /* picks per token */
    int32_t I;        /* routed expert intermediate size */
    int32_t SI;       /* shared expert intermediate size (0: none) */
    uint32_t flags;   /* MOE_LOGIT_OFFSET */
    float norm_eps;   /* latent RMSNorm epsilon */
} moe_latent_shape;

/* Workspace size of moe_latent_forward in *bytes (pure host function). */
int moe_latent_workspace_bytes(const moe_latent_shape* shape, size_t* bytes);

/*
 * The latent-MoE layer, all device pointers (16-byte aligned; w13, w2:
 * 32-byte aligned), enqueued on `stream`:
 *   x      [S, H] bf16           w_gate [E, H] bf16     bias [E] fp32
 *   logit_off [E] fp32 (MOE_LOGIT_OFFSET) or NULL
 *   w_ld   [LAT, H] bf16         latent down projection
 *   w13 [E, 2I, LAT/2], w13s [E, 2I, LAT/32], w2 [E, LAT, I/2], w2s
 *   [E, LAT, I/32]               the routed experts (MXFP4, as moe_experts)
 *   ln_w   [LAT] fp32            latent norm weight
 *   w_up   [H, LAT] bf16         up projection
 *   w_sgu  [2 SI, H] bf16        shared gate (rows 0..SI-1) and up rows
 *   w_sd   [H, SI] bf16          shared down (both NULL when SI == 0)
 *   ids, weights [S, k] out      the routing, as moe_route
 *   out    [S, H] fp32 out       overwritten
 * ws: at least moe_latent_workspace_bytes(), 256-byte aligned, prepared with
 * moe_workspace_init.  Errors as for moe_forward.
 */
int moe_latent_forward(const moe_latent_shape* shape, const void* x, const void* w_gate,
                       const float* bias, const float* logit_off, const void* w_ld,
                       const uint8_t* w13, const uint8_t* w13s,
                       const uint8_t* w2, const uint8_t* w2s,
                       const float* ln_w, const void* w_up,
                       const void* w_sgu, const void* w_sd,
                       int32_t* ids, float* weights, float* out,
                       void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------
 * The cache side of the verify step: what stands before the block in a layer.
 * One call feeds the next: moe_kv_plan (once a step) lays out where the new
 * tokens of every request go, moe_kv_append (a layer) writes their K and V rows
 * into the paged cache, moe_tree_attention (a layer) reads the cache.
 *
 * A batch holds B requests.  Request b has c_b = ctx_len[b] tokens in the cache
 * and brings n_b new ones: one token, a prompt or a part of one (a chain), or
 * a tree of drafted tokens.  The new tokens' rows of all requests stand one
 * after the other: request b owns rows row_start[b] .. row_start[b+1]-1, and
 * its row i is token c_b + i of its sequence in the cache.  Either count may be
 * zero.  The lengths are read on the device only, so no call waits for the GPU
 * and a captured graph serves any lengths that fit the shape.
 *
 * The cache is one K and one V tensor of pages of `page` tokens: element
 * (p, h, o, e) of either is at p * page_stride + h * head_stride +
 * o * token_stride + e.  Token a of request b is at offset a % page of page
 * block_table[b, a / page]; its slot is that page's id * page + a % page.
 * Entries are bf16, or with MOE_KV_E4M3 e4m3 codes (OCP 8-bit floating point)
 * that stand for code * scale, one positive fp32 scale a K/V head for K and one for V.
 */
#define MOE_KV_E4M3 1u  /* moe_kv_shape.flags: e4m3 cache */

/*
 * Supported: 1 <= B <= 4096; 1 <= T <= 1<<20; D 64 or 128; Hq a multiple of
 * Hkv with Hq / Hkv <= 128, Hq <= 4096; page a multiple of 8 up to 1024;
 * n_pages * page < 1<<31; max_pages * page <= 1<<30; 0 <= W <= 32; scale finite and > 0.
 * A stride of 0 is the packed one: cache [n_pages][Hkv][page][D], rows Hq * D and Hkv * D;
 * other strides are positive and cover a row (multiples of 16 bytes).
 */
typedef struct moe_kv_shape {
    int32_t B;             /* requests */
    int32_t T;             /* rows of new tokens the arrays hold */
    int32_t Hq, Hkv, D;    /* query heads, K/V heads, head width */
    int32_t page;          /* tokens a page */
    int32_t n_pages;       /* pages of the cache */
    int32_t max_pages;     /* columns of the block table */
    int32_t W;             /* 32-bit mask words a row; 0: chains, no mask */
    uint32_t flags;        /* MOE_KV_E4M3 */
    float scale;           /* factor of q . k before the softmax */
    int64_t page_stride, head_stride, token_stride;  /* cache, in elements */
    int64_t q_stride;      /* elements from one row of q to the next */
    int64_t kv_stride;     /* elements from one row of k_new (v_new) to the next */
} moe_kv_shape;

/*
 * Workspace size of the three calls in *bytes (pure host function).  Prepared
 * once with moe_workspace_init, and again after a MOE_ERR_TIMEOUT: counters in
 * it are 0 between calls, and a call that gave up leaves them as they were.
 * Calls that share a workspace must be ordered (one stream); errors found on
 * the device are reported by moe_device_status as for the block's calls.
 */
int moe_kv_workspace_bytes(const moe_kv_shape* shape, size_t* bytes);

/*
 * Block tables, slot maps, positions and tree masks from request lengths, in
 * one launch.  A request's pages are those its block-table row already holds
 * (the first ceil(c_b / page) entries) and then pages of the free list, taken
 * in request order.
 *   ctx_len, n_new [B]       int32
 *   parents   [T]            int32, or NULL (chains; W must be 0): the row of
 *                            its request a drafted token follows, an earlier
 *                            one, or -1 (it follows token c_b - 1)
 *   free_pages [n_free]      int32 page ids; a negative entry ends the list (may be
 *                            NULL when n_free is 0).  n_free is fixed in a captured
 *                            graph: the list itself then says how many there are,
 *                            with -1 in the places behind the last
 *   block_table [B, max_pages]  int32, in and out: entries ceil(c_b / page) ..
 *                            ceil((c_b + n_b) / page) - 1 are written
 *   row_start [B + 1]        int32 out
 *   slots     [T]            int64 out, positions [T] int32 out: c_b + the
 *                            depth in the tree (the row number in a chain);
 *                            both -1 in rows that no request owns
 *   mask      [T, W]         uint32 out (NULL when parents is): bit j % 32 of
 *                            word j / 32 of a row is set when row j of its
 *                            request is the row itself or an ancestor
 *   used      [2]            int32 out: rows owned, free pages taken
 * Device errors: MOE_ERR_BAD_LENGTHS (detail: the request; a negative length,
 * more tokens than the block table or, in a tree, the mask holds: the request
 * gets no rows; detail B: more than T rows, the last are cut off),
 * MOE_ERR_NO_PAGES (detail: pages missing; entries and slots are -1),
 * MOE_ERR_BAD_PARENT (detail: the row; its walk ends there), MOE_ERR_BAD_PAGE (detail:
 * the id; slots in that page are -1; also a negative entry of the list before a page id).
 */
int moe_kv_plan(const moe_kv_shape* shape, const int32_t* ctx_len, const int32_t* n_new,
                const int32_t* parents, const int32_t* free_pages, int32_t n_free,
                int32_t* block_table, int32_t* row_start, int64_t* slots, int32_t* positions,
                uint32_t* mask, int32_t* used, void* ws, size_t ws_bytes, void* stream);

/*
 * The new tokens' K and V rows into the cache: k_new, v_new [T, Hkv, D] bf16
 * (rows kv_stride apart) to slots [T] (distinct; a negative slot's row is
 * skipped, one past the cache is skipped and latches MOE_ERR_BAD_PAGE).
 * k_scale, v_scale [Hkv] fp32 with MOE_KV_E4M3 (else NULL): a code is
 * x / scale, rounded to nearest even and saturated at +-448.
 */
int moe_kv_append(const moe_kv_shape* shape, const void* k_new, const void* v_new, const int64_t* slots,
                  const float* k_scale, const float* v_scale, void* k_cache, void* v_cache,
                  void* ws, size_t ws_bytes, void* stream);

/*
 * Attention of the new tokens over the cache (which holds their own K and V
 * already).  Row i of request b sees the c_b cached tokens and those of its
 * request's new ones its mask row names (W = 0: rows 0..i).  For query head h
 * over K/V head h / (Hq / Hkv), with x_j = scale * q . k_j over the keys seen:
 *   lse = ln sum_j exp(x_j),   out = sum_j exp(x_j - lse) v_j
 * A row that sees nothing (a score of -inf counts as not seen) gets out 0 and
 * lse -inf; rows that no request owns are not written.  What a row does not
 * see does not reach it, whatever it holds (NaN included).  Sums and the softmax's maximum and
 * sum are fp32; the weights enter the second product as bf16.  With an e4m3 cache
 * the weights enter as f16 (11 bits for weights down to 2^-21 of the row's largest,
 * below that an error of at most 2^-32 of it), and q as two e4m3 terms under one power of
 * two a row: exact for elements down to 2^-9 of the row's largest, below that
 * with an error of at most 2^-17 of it.
 *   q [T, Hq, D] bf16 (rows q_stride apart); block_table [B, max_pages],
 *   ctx_len [B], row_start [B + 1], mask [T, W] (NULL when W is 0) as
 *   moe_kv_plan leaves them; k_scale, v_scale [Hkv] with MOE_KV_E4M3 (else
 *   NULL); out [T, Hq, D] bf16; lse [T, Hq] fp32 or NULL.
 * The launch's CTAs wait for one another: it needs the 152 SMs of a GB300, and
 * a device or context with fewer gets MOE_ERR_NO_DEVICE, with nothing enqueued.
 * Device errors: MOE_ERR_BAD_LENGTHS (detail: the request, which gets no
 * output), MOE_ERR_BAD_PAGE (detail: the id; that request's output is
 * unspecified), MOE_ERR_TIMEOUT.
 */
int moe_tree_attention(const moe_kv_shape* shape, const void* q, const void* k_cache, const void* v_cache,
                       const int32_t* block_table, const int32_t* ctx_len, const int32_t* row_start,
                       const uint32_t* mask, const float* k_scale, const float* v_scale,
                       void* out, float* lse, void* ws, size_t ws_bytes, void* stream);

/*
 * What stands between a fused query, key and value projection and the cache, in
 * one pass: an RMSNorm of each query and key head, the rotation by position,
 * and the append of K and V.  With x one head's row of D elements:
 *   y    = x * rsqrt(mean(x^2) + eps) * w          (w NULL: y = x)
 *   z_i  = y_i cos_i - y_j sin_i,  z_j = y_j cos_i + y_i sin_i
 * for the pairs (i, j) of the first R elements, i = 0 .. R/2 - 1: (i, i + R/2), or with
 * MOE_ROPE_INTERLEAVED elements 2i and 2i + 1; elements from R on are left as
 * they are.  cos_i and sin_i are entries i and R/2 + i of the table's row
 * positions[t].  Everything is fp32 and rounded once: q to bf16, K and V to the
 * cache's type as moe_kv_append does (V is neither normalised nor rotated).
 */
#define MOE_ROPE_INTERLEAVED 1u /* moe_rope.flags */

/*
 * Supported: R a multiple of 16, 0 (no rotation) to D; max_pos >= 1 when R > 0; eps
 * finite and >= 0; q_in_stride as q_stride of moe_kv_shape (0: packed).
 */
typedef struct moe_rope {
    int32_t R;             /* elements of a head that are rotated */
    int32_t max_pos;       /* rows of the table */
    uint32_t flags;        /* MOE_ROPE_INTERLEAVED */
    float eps;
    int64_t q_in_stride;   /* elements from one row of q_in to the next */
} moe_rope;

/*
 *   q_in [T, Hq, D] bf16 (rows q_in_stride apart); k_new, v_new [T, Hkv, D]
 *   bf16 (rows kv_stride apart): the three parts of a projection's rows, for
 *   instance.  positions [T] int32 and slots [T] int64 as moe_kv_plan leaves them.
 *   q_norm, k_norm [D] fp32, each may be NULL; cos_sin [max_pos, R] fp32
 *   (NULL when R is 0); k_scale, v_scale as for moe_kv_append.
 *   q [T, Hq, D] bf16 out (rows q_stride apart): q_in itself (then the
 *   strides have to be equal, else MOE_ERR_INVALID_ARG) or memory apart from it.
 * A row with a negative position is skipped; a row with a negative slot gets its
 * q but is not appended; slots are distinct.  Device errors: MOE_ERR_BAD_LENGTHS (detail:
 * the row; a position past the table, the row is skipped), MOE_ERR_BAD_PAGE
 * (detail: the page; a slot past the cache, the row is not appended).
 */
int moe_qkv_append(const moe_kv_shape* shape, const moe_rope* rope, const void* q_in, const void* k_new,
                   const void* v_new, const int32_t* positions, const int64_t* slots, const float* q_norm,
                   const float* k_norm, const float* cos_sin, const float* k_scale, const float* v_scale,
                   void* q, void* k_cache, void* v_cache, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------
 * Dense MXFP4: a layer's projections in the experts' weight format.  Rows are
 * packed as w13 and w2 are (see the top): codes [rows, K/2] and scale bytes [rows, K/32].
 * What a call writes stands apart from what it reads.
 */
#define MOE_BF16 0
#define MOE_F16  1
#define MOE_F32  2

/*
 * Rows to MXFP4 (OCP Microscaling v1.0): for every 32 elements of a row, with M the
 * largest magnitude, the scale is 2^(floor(log2 M) - 2), at least 2^-127 (byte 0,
 * also where M is 0); a code is x / scale rounded to nearest even and
 * saturated at +-6.  A block that holds a NaN or an infinity gets scale byte
 * 255 and codes 0: it reads back as NaN.
 *   x [rows, K] of type dtype (MOE_BF16, MOE_F16, MOE_F32), rows x_stride elements apart
 *   (0: K; rows multiples of 16 bytes apart); codes and scales out, packed.
 * K a multiple of 32 up to 1<<20; 1 <= rows, rows * K < 1<<44.  No workspace.
 */
int moe_mx_quantize(int64_t rows, int32_t K, int dtype, const void* x, int64_t x_stride, uint8_t* codes,
                    uint8_t* scales, void* stream);

/*
 * MXFP4 rows to y [rows, K] of type dtype, rows y_stride elements apart (as
 * above): code * scale, exact in fp32 (an infinity past its range, NaN under byte
 * 255) and rounded to the type (to nearest even).
 */
int moe_mx_dequantize(int64_t rows, int32_t K, int dtype, const uint8_t* codes, const uint8_t* scales, void* y,
                      int64_t y_stride, void* stream);

#define MOE_MX_X_MXFP4 1u /* moe_mx_shape.flags: x is MXFP4 too */

/*
 * out = x . w^T.  Supported: 1 <= T <= 1<<20; N a multiple of 8, 8 <= N <= 1<<20; K a
 * multiple of 128, 128 <= K <= 65536.  A stride of 0 is the packed one; others
 * cover a row and are multiples of 8 elements (x_stride: bf16 x only).
 */
typedef struct moe_mx_shape {
    int32_t T;           /* rows of x */
    int32_t N;           /* rows of w: columns of out */
    int32_t K;           /* length of the sums */
    uint32_t flags;      /* MOE_MX_X_MXFP4 */
    int64_t x_stride;    /* elements from one row of x to the next */
    int64_t out_stride;  /* ... of out */
} moe_mx_shape;

/*
 * Workspace size of moe_mx_linear in *bytes (pure host function); moe_workspace_init prepares it once.
 * The same for every N, and never less for more rows or a larger K: the workspace of a program's
 * largest T and K with a bf16 x serves all of its calls.
 */
int moe_mx_workspace_bytes(const moe_mx_shape* shape, size_t* bytes);

/*
 *   out[t, n] = sum_k x[t, k] * w[n, k], summed in fp32, rounded to bf16
 *   x [T, K] bf16, or with MOE_MX_X_MXFP4 codes [T, K/2] and xs [T, K/32]
 *   (xs NULL otherwise); w [N, K/2] codes (32-byte aligned), w_scales [N, K/32];
 *   out [T, N] bf16
 * The products are exact in fp32 but for a bf16 x, whose elements enter as two
 * e4m3 terms under a power of two a block of 32 (see the top): exact down to
 * 2^-9 of the block's largest magnitude, below that within 2^-17 of it.  Sums whose
 * magnitude is below 2^-126 may come out as 0.  A row of x
 * with a NaN or an infinity (MXFP4: a scale byte of 255) gives a row of NaN.
 * Device errors: MOE_ERR_BAD_SCALE (a scale byte of 255 in w: its column of out
 * is NaN), MOE_ERR_TIMEOUT (the workspace is then prepared again).
 * Calls that share a workspace must be ordered, as for the block's calls.
 */
int moe_mx_linear(const moe_mx_shape* shape, const void* x, const uint8_t* xs, const uint8_t* w,
                  const uint8_t* w_scales, void* out, void* ws, size_t ws_bytes, void* stream);

/*
 * How moe_mx_linear cuts a shape's work (diagnostics, pure host function; each pointer may be NULL): the CTAs
 * (1, or 2 for a pair) and the tokens of a tile, and how many CTAs of a cluster share a tile's K.
 */
int moe_mx_linear_cut(const moe_mx_shape* shape, int32_t* ctas, int32_t* tokens, int32_t* parts);

/*
 * Synchronises `stream`, returns the status latched in the workspace by the
 * device since the last call (MOE_OK, MOE_ERR_BAD_IDS, MOE_ERR_BAD_SCALE,
 * MOE_ERR_TIMEOUT or what the cache calls name; MOE_ERR_CUDA if the synchronisation itself failed) and
 * clears it.  *detail (may be NULL) receives a code-specific value: the first
 * offending flat pick index, the first bad scale byte's value, the site of
 * the wait that ran out, or what the cache calls name.
 */
int moe_device_status(void* ws, int32_t* detail, void* stream);

/*
 * Workspace regions (diagnostics, pure host function): byte offset and size
 * of one region of the workspace of `shape`, for reading intermediate results
 * back after a call (tests and profiling).  Returns MOE_OK, or
 * MOE_ERR_INVALID_ARG / MOE_ERR_UNSUPPORTED_SHAPE.  P = S * k picks; a pick's
 * sorted position r groups the picks by ascending expert id (k3 page,
 * dn_loads: tasks over a table of the experts that have picks).
 *   MOE_WS_STATUS  int32 [64]: status, detail, valid picks, work tiles, ...
 *   MOE_WS_POS     int32 [P]: sorted position r of pick t*k + j (-1: invalid)
 *   MOE_WS_TILES   int32 [max tiles][4]: expert, first position, picks, 0;
 *                  the first "work tiles" entries are this call's tiles
 *   MOE_WS_XQ      uint8 [2P][d]: e4m3 rows 2r (hi) and 2r + 1 (lo) of the
 *                  token of the pick at position r
 *   MOE_WS_XS      uint8 [ceil(d/256)][P + 64][16]: e8m0 scale of 32-element
 *                  block b of position r at [b / 8][r][b % 8]
 *   MOE_WS_HQ, MOE_WS_HS  the same for h = silu(g) * u (K = I)
 *   MOE_WS_Y       fp32 [P][d]: expert output of the pick at position r
 *   MOE_WS_LOGITS  fp32 [S][E]: the router's logits (moe_route, moe_forward)
 */
#define MOE_WS_STATUS 0
#define MOE_WS_POS    1
#define MOE_WS_TILES  2
#define MOE_WS_XQ     3
#define MOE_WS_XS     4
#define MOE_WS_HQ     5
#define MOE_WS_HS     6
#define MOE_WS_Y      7
#define MOE_WS_LOGITS 8
int moe_workspace_region(const moe_shape* shape, int region, size_t* offset, size_t* bytes);

/*
 * Per-kernel timing (diagnostics, host side).  After moe_timing_enable(n) with
 * n > 0, the next n kernels the library launches are each bracketed by a pair
 * of CUDA events recorded on their launch stream; n = 0 turns this off and
 * frees the events.  moe_timing_collect waits for the recorded events and
 * writes up to `cap` (kernel id, milliseconds) pairs in launch order, the
 * count to *n, and starts a new recording of the same size.  Kernel ids name
 * the launched kernels (moe_kernel_name; NULL past the last id).  Not
 * thread-safe; event records add a few microseconds of host time per launch.
 * Returns MOE_OK, MOE_ERR_INVALID_ARG or MOE_ERR_CUDA.
 */
int moe_timing_enable(int max_launches);
int moe_timing_collect(int32_t* kernel_ids, float* ms, int cap, int* n);
const char* moe_kernel_name(int kernel_id);

#ifdef __cplusplus
}
#endif

#endif /* MOE_H */
