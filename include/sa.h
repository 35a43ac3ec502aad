/*
 * sa.h -- C ABI of the GB300 (sm_103a) routed block-sparse self-attention
 * library (libsa_gb300.so).
 *
 * The layer: one packed sequence per batch entry, [B, S, H, D] bf16 Q/K/V
 * ("MiniMax H3 runs on single 4090 with 4.44x speedup over dense execution",
 * third paragraph: [1, 38247, 56, 128], tau = 1.0, diagonal, exact prefix
 * KV sink, compressed prefix queries; Sol-Engine H3-DataCenter release page,
 * policy paragraph: a 951-token exact prefix sink, no token reordering, the
 * first steps and layers dense).
 *
 * Conventions shared by every entry point:
 *  - Device pointers are device memory of the current CUDA device; host
 *    pointers are named *_host. The caller owns every buffer. The library
 *    never allocates device memory, frees or synchronises: every call
 *    enqueues work on `stream` (a cudaStream_t passed as void*; NULL = the
 *    legacy default stream) and returns (sa_forward_host also uses two copy
 *    streams of its own, see there).
 *  - The returned sa_status reports what can be checked before launch
 *    (arguments, support, launch errors). Conditions found on the device are
 *    OR-ed into *dev_status (an int32 in device memory that the caller sets
 *    to 0 before the first call and reads after the stream; NULL = do not
 *    report) as SA_DEV_* bits. The kernels never trap.
 *  - Tensors are [B, S, H, D] with the d index contiguous; the strides for
 *    b, s and h are given in elements and must be multiples of 8 (16 bytes),
 *    and every tensor base must be 16-byte aligned.
 *  - Query and key blocks are contiguous 64-token ranges; Nb = ceil(S/64);
 *    the last block holds S - 64 (Nb - 1) valid tokens. Tokens at or beyond S
 *    never contribute (the padding contributes exactly zero: "Making
 *    MiniMax-H3 up to 9x faster on H100s", section "The benchmark was not the
 *    product").
 */
#ifndef SA_GB300_H
#define SA_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum sa_status {
  SA_OK = 0,
  SA_ERR_INVALID_ARG = 1, /* a NULL pointer, a bad size, stride or alignment   */
  SA_ERR_UNSUPPORTED = 2, /* a valid request this build does not serve (D)     */
  SA_ERR_CAPACITY = 3,    /* a buffer or workspace is smaller than required    */
  SA_ERR_CUDA = 4,        /* a CUDA runtime or driver call failed              */
  SA_ERR_TIMEOUT = 5      /* (decoded from dev_status) a bounded wait expired  */
} sa_status;

/* Bits OR-ed into *dev_status by the kernels. */
enum {
  SA_DEV_CAPACITY = 1 << 0, /* the route had more than col_cap entries; the
                               CSR is truncated (row_ptr is still exact)      */
  SA_DEV_TIMEOUT = 1 << 1,  /* a bounded pipeline wait gave up; the output of
                               the affected tiles is undefined                */
  SA_DEV_BAD_ROUTE = 1 << 2,/* sa_attn_sparse met a CSR that breaks its
                               contract (see sa_attn_sparse for what is then
                               attended)                                      */
  SA_DEV_RANGE = 1 << 3,    /* a V value does not fit fp16 (|v| > 65504); the
                               P.V product runs in fp16, see sa_attn_sparse    */
  SA_DEV_BAD_CACHE = 1 << 4,/* a paged-cache call met a sequence length or a
                               page id outside its range (see sa_cache_params
                               for what is then done)                         */
  SA_DEV_BAD_TREE = 1 << 5  /* a new token's parent that does not come before
                               it (sa_attn_tree), a path that does not ascend
                               (sa_cache_accept) or a source row that does not
                               exist (sa_pages_fork); see there               */
};

/* Arithmetic of the attention's score product Q.K^T (sa_attn_*). */
enum {
  SA_QK_BF16 = 0,   /* bf16 x bf16 -> fp32 (the default)                       */
  SA_QK_FP8 = 1     /* 8-bit scores: Q and K quantised to e4m3 per (batch,
                       head, 64-token block) with power-of-two scales, see
                       sa_qk_quantize; D = 128 only                           */
};

/* Readings of the router rule (sa_route; the pages leave the rule open). */
enum {
  SA_ROUTE_THRESHOLD = 0,           /* keep p_ij >= tau / Nb (the default)     */
  SA_ROUTE_DENSE_PREFIX_QUERIES = 1,/* as THRESHOLD, and every query block that
                                       meets the prefix keeps every key block */
  SA_ROUTE_TOP_MASS = 2             /* keep the fewest key blocks of largest
                                       p_ij whose summed p_ij reaches tau     */
};

typedef struct sa_params {
  int32_t B, S, H, D;     /* D must be 64 or 128; B, S, H >= 1               */
  int32_t block;          /* must be 64                                       */
  int32_t prefix_len;     /* P, 0 <= P <= S: key tokens [0, P) are always
                             attended, via every key block j < ceil(P/64)    */
  float tau;              /* router parameter, >= 0: for THRESHOLD and
                             DENSE_PREFIX_QUERIES a multiple of the uniform
                             share (0 keeps every block); for TOP_MASS a mass
                             in [0, 1] (0 keeps only the forced blocks)      */
  float softmax_scale;    /* 0 => 1/sqrt(D); used for routing and attention  */
  int64_t q_stride[3];    /* element strides of b, s, h (d is contiguous)    */
  int64_t k_stride[3];
  int64_t v_stride[3];
  int64_t o_stride[3];
  int32_t route_mode;     /* SA_ROUTE_*; sa_params_init sets THRESHOLD       */
  int32_t q_block;        /* query block of the route: 0 or 64 (square, the
                             default) or 128 (two key blocks); see sa_route  */
  int32_t qk_format;      /* SA_QK_*; sa_params_init sets SA_QK_BF16         */
} sa_params;

/* Fills p for a contiguous [B, S, H, D] layout of all four tensors, with
 * route_mode = SA_ROUTE_THRESHOLD, q_block = 0, qk_format = SA_QK_BF16 and
 * softmax_scale = 0. */
void sa_params_init(sa_params* p, int32_t B, int32_t S, int32_t H, int32_t D,
                    int32_t prefix_len, float tau);

/* Nb = ceil(S / 64) (0 on bad params). */
int32_t sa_num_blocks(const sa_params* p);

/* Number of CSR rows, B*H*Nb; row_ptr holds this + 1 entries. */
int64_t sa_route_rows(const sa_params* p);

/* Worst-case number of route entries, B*H*Nb*Nb (every block kept). */
int64_t sa_route_max_nnz(const sa_params* p);

/* Bytes of device workspace sa_route needs (256-byte aligned start). */
size_t sa_route_workspace_bytes(const sa_params* p);

/*
 * sa_route -- the online router: for every (b, h, query block i) the
 * ascending list of key blocks that query block i attends.
 *
 * Rule (the pages name an online router with threshold tau over compressed
 * queries and keys, a diagonal threshold and an exact prefix sink; the exact
 * formula is this library's reading of them):
 *   qbar_i, kbar_j = mean of the valid Q / K tokens of block i / j;
 *   s_ij = softmax_scale * qbar_i . kbar_j for every key block j;
 *   p_ij = softmax over j of s_ij;
 *   keep j  iff  p_ij >= tau / Nb,  or j < ceil(P/64) (sink),  or j == i.
 * p->route_mode selects another reading: DENSE_PREFIX_QUERIES also keeps
 * every key block of query blocks i < ceil(P/64); TOP_MASS replaces the
 * first test by: rank the key blocks by p_ij descending (equal p_ij: lower j
 * first) and keep block j iff the blocks ranked above it sum to less than
 * tau.
 * p->q_block = 128 (any mode) routes 128-token query blocks over the same
 * 64-token key blocks: qbar_i is the mean of the valid tokens of query
 * tokens [128 i, 128 i + 128), the threshold is still tau / Nb with Nb the
 * number of key blocks, the diagonal of query block i is key blocks 2i and
 * 2i + 1, and DENSE_PREFIX_QUERIES covers query blocks i < ceil(P/128). The
 * CSR keeps one row per 64-token block: rows 2i and 2i + 1 both hold query
 * block i's list, so sa_attn_sparse reads it unchanged.
 * Decisions match an fp64 evaluation of the rule except on ties: for
 * THRESHOLD, |p_ij * Nb / tau - 1| <= 1e-6; for TOP_MASS, a preceding mass
 * within 1e-6 of tau, or p_ij within a relative 1e-6 of the last kept
 * block's across the cut. Pooling is exact to fp64 rounding; the scores are computed in fp32
 * and every row holding a decision inside a rigorous fp32 error bound is
 * recomputed in fp64.
 *
 * q, k       device, bf16 [B, S, H, D] with the strides in p; not modified.
 * row_ptr    device int32 [B*H*Nb + 1]; row r = (b*H + h)*Nb + i.
 *            row_ptr[0] = 0, row_ptr[r+1] - row_ptr[r] = entries of row r.
 * col_idx    device int32 [col_cap]; the key blocks of row r, ascending, at
 *            col_idx[row_ptr[r] .. row_ptr[r+1]).
 * col_cap    capacity of col_idx. If the route is longer, entries beyond
 *            col_cap are dropped and SA_DEV_CAPACITY is raised; passing
 *            sa_route_max_nnz(p) can never overflow.
 * workspace  device scratch of at least sa_route_workspace_bytes(p) bytes,
 *            256-byte aligned; its contents on entry do not matter.
 * Errors: SA_ERR_INVALID_ARG / SA_ERR_UNSUPPORTED / SA_ERR_CAPACITY (ws
 * too small) before launch; SA_ERR_CUDA if a launch fails.
 */
sa_status sa_route(const sa_params* p, const void* q, const void* k,
                   int32_t* row_ptr, int32_t* col_idx, int64_t col_cap,
                   void* workspace, size_t ws_bytes, int32_t* dev_status,
                   void* stream);

/* Size of the library-owned device scratch array sa_route_static runs on. */
#define SA_ROUTE_STATIC_WS_BYTES (32u << 20) /* 32 MiB */

/*
 * sa_route_static -- sa_route for callers that cannot allocate device
 * memory. The pages have no counterpart to this entry point; it exists for
 * callers such as a plugin inside an inference engine that has already
 * reserved all of HBM for its own pool, or code on a latency-critical path
 * where a cudaMalloc would synchronise the device.
 *
 * It computes exactly what sa_route computes (same kernels, same result) but
 * takes no workspace: the scratch lives in a fixed device array of
 * SA_ROUTE_STATIC_WS_BYTES inside the library, which every GPU that loads
 * the library holds until the process exits. It allocates nothing and frees
 * nothing. The caller still passes q, k, row_ptr, col_idx (as for sa_route).
 *
 * Limits and behaviour:
 *  - Shapes whose sa_route_workspace_bytes(p) exceeds SA_ROUTE_STATIC_WS_BYTES
 *    are rejected with SA_ERR_CAPACITY before anything is launched. With
 *    D = 128 and 64-token query blocks the limit is 9 heads at S = 38,247,
 *    72 at S = 8,192 and 1 at S = 112,640 (15, 101 and 3 heads with
 *    q_block = 128); sa_route_workspace_bytes gives the need of any shape.
 *  - The first call on each device, made with that device current, looks up
 *    the array's device address and caches it; make that first call before
 *    any stream capture.
 *  - Every call on a device uses the same array and finds the previous call's
 *    contents there; what must start at zero is cleared by each call. Calls
 *    whose work overlaps on the GPU (e.g. on two unordered streams) race on
 *    the array and give undefined routes: order them on one stream.
 * Errors: as sa_route, plus SA_ERR_CAPACITY for shapes beyond the limit and
 * SA_ERR_CUDA if the array's address cannot be obtained.
 */
sa_status sa_route_static(const sa_params* p, const void* q, const void* k,
                          int32_t* row_ptr, int32_t* col_idx, int64_t col_cap,
                          int32_t* dev_status, void* stream);

/*
 * sa_qk_prologue -- QK-norm + RoPE of q and k with the router's pooling
 * fused in (the fused QK-norm plus RoPE kernel of "Making MiniMax-H3 up to
 * 9x faster on H100s", section "Custom kernels"; the formulas are this
 * library's reading of that step). For every (b, token t, h) vector x [D]
 * of q_in (weights gamma_q) and of k_in (weights gamma_k):
 *   y_d = x_d / sqrt(mean_d(x_d^2) + eps) * gamma_d
 *   (y_2i, y_2i+1) -> (y_2i c - y_2i+1 s, y_2i s + y_2i+1 c),
 *       c = rope_cos[t][i], s = rope_sin[t][i]
 * computed in fp32 and rounded once to bf16 into q_out / k_out. The block
 * means of those bf16 outputs are written into `workspace` exactly as
 * sa_route would compute them from q_out, k_out; sa_route_pooled then
 * routes from them, so q_out and k_out are not read again for routing.
 *
 * q_in, k_in   device bf16 [B, S, H, D], strides p->q_stride / p->k_stride.
 * q_out, k_out device bf16, the same strides as q_in / k_in; each may be
 *              the same buffer as its input (in place) but must not
 *              otherwise overlap it.
 * gamma_q,     device fp32 [D], 16-byte aligned, or NULL for all ones.
 * gamma_k
 * eps          >= 0, added to the mean square.
 * rope_cos,    device fp32 [S][D/2] (row t = token t of the packed
 * rope_sin     sequence, any 1-D or 3-D rotary scheme), 16-byte aligned;
 *              both NULL for no rotation.
 * workspace    the route workspace, sa_route_workspace_bytes(p) bytes,
 *              256-byte aligned; p->q_block sets the query pooling.
 * Errors: as sa_route (SA_ERR_INVALID_ARG also for a bad eps, an unaligned
 * weight or table, or only one of the two tables).
 */
sa_status sa_qk_prologue(const sa_params* p, const void* q_in, const void* k_in,
                         const float* gamma_q, const float* gamma_k, float eps,
                         const float* rope_cos, const float* rope_sin, void* q_out,
                         void* k_out, void* workspace, size_t ws_bytes,
                         int32_t* dev_status, void* stream);

/* A pair that sa_rope_axes leaves as it is. */
#define SA_ROPE_STAYS 255

/* Rotary positions with several axes (time, height, width): pair i of a head
 * vector is turned by row `position on axis axis_of[i]` of the rotation tables,
 * column i. A pair of SA_ROPE_STAYS is not turned, whatever it holds. */
typedef struct sa_rope_axes {
  const int32_t* positions; /* device int32 [B][S][n_axes], the axes contiguous,
                               or NULL: a token's place in its sequence, on
                               every axis                                      */
  int64_t pos_stride[2];    /* elements between two sequences, two tokens     */
  int32_t n_axes;           /* 1 to 8                                          */
  int32_t rows;             /* rows of the rotation tables, >= 1. A position
                               outside [0, rows) counts as the nearest one
                               inside and raises SA_DEV_CAPACITY               */
  uint8_t axis_of[64];      /* of pair i < D/2: an axis, or SA_ROPE_STAYS      */
} sa_rope_axes;

/*
 * sa_qk_prologue_axes -- sa_qk_prologue with positions on several axes: token t
 * of sequence b turns pair i by rope_cos, rope_sin[positions[b][t][axis_of[i]]][i].
 * The tables hold every position once, not every token. qk_norm = 0 leaves the
 * norm out (the gammas are then NULL); rope_cos and rope_sin (fp32
 * [axes->rows][D/2]) are given. Else, the block means that sa_route_pooled routes
 * from among it, as sa_qk_prologue.
 */
sa_status sa_qk_prologue_axes(const sa_params* p, const void* q_in, const void* k_in,
                              int32_t qk_norm, const float* gamma_q, const float* gamma_k,
                              float eps, const float* rope_cos, const float* rope_sin,
                              const sa_rope_axes* axes, void* q_out, void* k_out,
                              void* workspace, size_t ws_bytes, int32_t* dev_status,
                              void* stream);

/*
 * sa_route_pooled -- sa_route from the block means that sa_qk_prologue left
 * in `workspace` (steps after pooling: logits, selection, fp64 recheck,
 * CSR). p must give the same B, S, H, D, q_block and strides as that
 * sa_qk_prologue call (prefix_len, tau, route_mode and softmax_scale may
 * differ); the workspace's contents are not checked. The result equals
 * sa_route on the prologue's q_out, k_out. Arguments and errors as sa_route.
 */
sa_status sa_route_pooled(const sa_params* p, int32_t* row_ptr, int32_t* col_idx,
                          int64_t col_cap, void* workspace, size_t ws_bytes,
                          int32_t* dev_status, void* stream);

/*
 * sa_qk_quantize -- the 8-bit copies of q and k that sa_attn_* use with
 * p->qk_format = SA_QK_FP8 (MiniAcc blog, "What is SageAttention?": the
 * score computation in 8-bit arithmetic; the format and scaling are this
 * library's reading: FP8 e4m3, the 8-bit format GB300's tensor cores run
 * fastest). For every (b, h, 64-token block j) of q, and of k:
 *   e     = the smallest integer with amax / 2^e <= 448, where amax is the
 *           largest |x| over the block's valid tokens and all D (e = 0 for
 *           an all-zero block);
 *   code  = x / 2^e rounded to the nearest e4m3 value, ties to even
 *           (exact scaling: the scale is a power of two).
 * The attention's logits are then scale * 2^(e_q + e_k) * (codes_q . codes_k).
 *
 * q, k          device bf16 [B, S, H, D] (strides in p), D = 128.
 * q8, k8        device uint8 [B, S, H, D], contiguous, 8-byte aligned: the
 *               e4m3 codes (tokens >= S are not written).
 * q_exp, k_exp  device int8 [B*H*Nb]: e of block (b, h, j) at (b*H + h)*Nb + j.
 * A non-finite input raises SA_DEV_RANGE (its block's codes are undefined).
 * Errors: SA_ERR_INVALID_ARG / SA_ERR_UNSUPPORTED (D != 128) before launch.
 */
sa_status sa_qk_quantize(const sa_params* p, const void* q, const void* k, uint8_t* q8,
                         uint8_t* k8, int8_t* q_exp, int8_t* k_exp, int32_t* dev_status,
                         void* stream);

/* Bytes of device workspace sa_attn_sparse / sa_attn_dense need (more with
 * p->qk_format = SA_QK_FP8: the codes of Q and K live there). */
size_t sa_attn_workspace_bytes(const sa_params* p);

/*
 * sa_attn_sparse -- block-sparse attention forward over a route: only the
 * routed (query block, key block) pairs are computed (MiniAcc blog, "What is
 * Sol attention?"), each exactly (exact softmax over the selected keys).
 *
 * For every query token t of block i (head h, batch b), over the valid key
 * tokens u of the key blocks listed for row (b, h, i):
 *   l_u = softmax_scale * q_t . k_u,   a_u = exp(l_u - max l) / sum exp(.),
 *   o_t = sum_u a_u v_u,              lse_t = max l + log sum exp(l - max l).
 * Only the listed K/V blocks are read. A row with an empty list gives o = 0
 * and lse = -inf.
 *
 * Precision: Q.K^T is a bf16 x bf16 product with fp32 accumulation (with
 * p->qk_format = SA_QK_FP8: an e4m3 x e4m3 product of sa_qk_quantize's codes,
 * fp32 accumulation, times the blocks' power-of-two scales; the codes are
 * made in the workspace by each call); the softmax is fp32; the P.V product
 * takes P and V in fp16 (V is repacked once per call into the workspace)
 * with fp32 accumulation; o is rounded once to bf16. |v| must be <= 65504
 * (else SA_DEV_RANGE).
 *
 * q, k, v    device bf16 [B, S, H, D] (strides in p); not modified.
 * row_ptr,   device int32 CSR as written by sa_route: row_ptr[B*H*Nb] = nnz
 * col_idx    entries in col_idx (which must hold at least that many), each
 *            row strictly ascending with entries in [0, Nb). A CSR that
 *            breaks this raises SA_DEV_BAD_ROUTE and is attended as follows:
 *            a row whose span [row_ptr[r], row_ptr[r+1]) does not lie inside
 *            [0, nnz] or is longer than Nb is skipped whole (its query rows
 *            give o = 0, lse = -inf; col_idx is not read for it); entries
 *            outside [0, Nb) are skipped; a row that is not strictly
 *            ascending (a repeated entry included) is attended as the set of
 *            its entries. Nothing is read outside col_idx[0, nnz).
 * o          device bf16 [B, S, H, D] (o_stride); rows >= S are not written.
 * lse        device fp32 [B, H, S] (natural log), or NULL.
 * workspace  device scratch of sa_attn_workspace_bytes(p) bytes, 256-byte
 *            aligned.
 * Each 128-row tile of the kernel holds two 64-token query blocks of one
 * head. With p->q_block = 0 or 64 the pairs are chosen per call from the
 * route (largest key-list overlap, among blocks at most 32 apart); with
 * p->q_block = 128 the tiles are the 128-token query blocks (2i, 2i + 1),
 * which share their key list when the route came from sa_route with the
 * same q_block (any CSR is still attended exactly).
 */
sa_status sa_attn_sparse(const sa_params* p, const void* q, const void* k,
                         const void* v, const int32_t* row_ptr,
                         const int32_t* col_idx, void* o, float* lse,
                         void* workspace, size_t ws_bytes, int32_t* dev_status,
                         void* stream);

/*
 * sa_attn_prepare, sa_attn_run -- sa_attn_sparse in two calls, with the same
 * result: sa_attn_prepare repacks V into the workspace and (for 64-token
 * query blocks) chooses the tile pairs from the route; sa_attn_run launches
 * the attention kernel over that workspace (with SA_QK_FP8, after quantising
 * q and k into it, as sa_qk_quantize does). Between them the caller may
 * enqueue other work (or time the kernel alone); sa_attn_run must see the
 * same p, route and workspace, after sa_attn_prepare on the same stream (or
 * ordered after it), and V unchanged. Arguments and errors as
 * sa_attn_sparse, each call checking what it takes.
 */
sa_status sa_attn_prepare(const sa_params* p, const void* v, const int32_t* row_ptr,
                          const int32_t* col_idx, void* workspace, size_t ws_bytes,
                          int32_t* dev_status, void* stream);
sa_status sa_attn_run(const sa_params* p, const void* q, const void* k,
                      const int32_t* row_ptr, const int32_t* col_idx, void* o, float* lse,
                      void* workspace, size_t ws_bytes, int32_t* dev_status, void* stream);

/*
 * sa_attn_dense -- the same forward with every key block attended (density
 * 100%), as the pages run for the first denoising steps and the first layers
 * (Sol-Engine H3-DataCenter release page, policy paragraph). Arguments as in
 * sa_attn_sparse, without the route.
 */
sa_status sa_attn_dense(const sa_params* p, const void* q, const void* k,
                        const void* v, void* o, float* lse, void* workspace,
                        size_t ws_bytes, int32_t* dev_status, void* stream);

/*
 * sa_forward_host -- one whole layer from host memory: copies q, k, v
 * (host, pinned for asynchronous copies) to the device buffers, routes,
 * attends, and copies o (and lse if both lse pointers are non-NULL) back,
 * then returns without synchronising. The work is split into groups of
 * heads (for H >= 16 five groups, a quarter of the heads each and then a
 * seventh and the rest, since wide head slices copy faster and narrow last
 * groups shorten the tail; one group for H < 16 or for B > 1 with lse):
 * each group is routed and attended as soon as its q, k, v slices have
 * landed, and its o slice is copied back as soon as it is done, so the
 * copies overlap the compute. Compute runs on `stream`; the copies run on two
 * streams the library creates, with a few events, on the first call on each
 * device and keeps until the process exits. All of it is ordered after the
 * work enqueued on `stream` before the call and before the work enqueued on
 * it after the call. Calls on one device from several host threads are
 * serialised by the library. Every device buffer is the caller's, sized as
 * for sa_route / sa_attn_sparse, with q_dev, k_dev, v_dev, o_dev laid out
 * with the strides in p and *_host contiguous copies of the same
 * [B, S, H, D] extents (the strides in p must then describe a contiguous
 * tensor). The route workspace and the attention workspace may be the same
 * buffer if it is large enough for both.
 */
sa_status sa_forward_host(const sa_params* p, const void* q_host,
                          const void* k_host, const void* v_host, void* o_host,
                          float* lse_host, void* q_dev, void* k_dev,
                          void* v_dev, void* o_dev, float* lse_dev,
                          int32_t* row_ptr, int32_t* col_idx, int64_t col_cap,
                          void* workspace, size_t ws_bytes,
                          int32_t* dev_status, void* stream);

/*
 * sa_check_wait_timeout -- a device check of the failure path that every
 * pipeline wait of this library shares (no counterpart on the pages): it
 * launches one warp that waits on a barrier nothing completes. The wait gives
 * up after the library's time limit (250 ms), OR-s SA_DEV_TIMEOUT into
 * *dev_status (device memory, required) and the kernel returns; the context
 * stays usable. Nothing faults, traps or hangs. Asynchronous on `stream`.
 */
sa_status sa_check_wait_timeout(int32_t* dev_status, void* stream);

/* ------------------------------------------------------------------------
 * The paged key-value cache: keys and values that stay between calls, and the
 * attention of one new token over them. (The pages attend one whole packed
 * sequence per call and have no counterpart; the key blocks, the pooled keys,
 * the sink, the diagonal and the list format are those of the layer above.)
 *
 * A cache is a pool of pages of 64 tokens, the library's key block:
 *   k_cache, v_cache  [n_pages, H_kv, 64, D] bf16 or e4m3, d contiguous, with
 *                     any strides of page, head and token;
 *   page_table        int32 [B, max_pages]: token t of sequence b lives in
 *                     page page_table[b][t / 64], slot t % 64;
 *   seq_lens          int32 [B], device memory: the tokens of each sequence;
 *   k_sum             fp32 [n_pages, H_kv, D], contiguous: the sum of a page's
 *                     keys, which ranks pages as sa_route's block means do
 *                     (only the router needs it).
 * H query heads share H_kv key-value heads, H / H_kv consecutive ones each.
 *
 * Nothing is read or written outside these extents: a length below 0 counts as
 * 0, one beyond 64 max_pages as 64 max_pages, and the tokens of a page whose
 * id is outside [0, n_pages) are left out; each raises SA_DEV_BAD_CACHE.
 * Entries of page_table behind a sequence's last page are not read. One page
 * may serve several sequences or places as long as nothing is appended to it;
 * what a page holds that is appended to in two places in one call is undefined.
 *
 * Lengths, tables and routes are read when the call runs, so a captured call
 * serves as they change; they must not change while it runs. Calls that may run
 * at the same time need workspaces of their own.
 * ---------------------------------------------------------------------- */

/* Storage of the cached keys and values. */
enum {
  SA_CACHE_BF16 = 0,
  SA_CACHE_FP8 = 1   /* e4m3; value = code * scale of its key-value head       */
};

/* Which two elements of a head vector the rotation turns together. */
enum {
  SA_ROPE_INTERLEAVED = 0, /* 2i and 2i + 1, as sa_qk_prologue (the default)  */
  SA_ROPE_HALF = 1         /* i and i + D/2                                    */
};

typedef struct sa_cache_params {
  int32_t B, S, H, H_kv, D; /* S: new tokens per sequence (1 where one new
                               token attends or is routed); H % H_kv == 0;
                               D must be 64 or 128                             */
  int32_t page;             /* must be 64                                      */
  int32_t n_pages;          /* pages of the pool, >= 1                         */
  int32_t max_pages;        /* page-table entries of a sequence, >= 1 and
                               < 2^25                                          */
  int32_t cache_format;     /* SA_CACHE_*                                      */
  int32_t prefix_len;       /* sa_route_pages: P >= 0, as sa_params           */
  int32_t page_budget;      /* sa_route_pages: pages to keep, >= 0            */
  int32_t qk_norm;          /* sa_cache_append: 0 or 1                         */
  int32_t rope_layout;      /* sa_cache_append: SA_ROPE_*                      */
  int32_t rope_rows;        /* sa_cache_append: rows of the rotation tables    */
  float eps;                /* sa_cache_append: >= 0, added to the mean square */
  float softmax_scale;      /* sa_attn_decode, _tree: 0 => 1/sqrt(D)           */
  int64_t table_stride;     /* elements between two sequences of page_table    */
  int64_t q_stride[3];      /* element strides of b, s, h of the new tokens'   */
  int64_t k_stride[3];      /* q, k, v and of o (sa_cache_append: of q_out),   */
  int64_t v_stride[3];      /* multiples of 8 as in sa_params                  */
  int64_t o_stride[3];
  int64_t kc_stride[3];     /* element strides of page, head, token of the     */
  int64_t vc_stride[3];     /* caches: multiples of 16 bytes                   */
} sa_cache_params;

/* Fills p for contiguous tensors and caches in bf16: page = 64, S = 1,
 * table_stride = max_pages, eps = 1e-6, the rest 0. */
void sa_cache_params_init(sa_cache_params* p, int32_t B, int32_t H, int32_t H_kv, int32_t D,
                          int32_t n_pages, int32_t max_pages);

/*
 * sa_cache_append -- the new tokens' keys and values into the cache, with
 * QK-norm and rotation on the way (the step sa_qk_prologue makes for a whole
 * packed sequence). Token s < n_b of sequence b (n_b = new_lens[b], S where
 * new_lens is NULL) takes position t = seq_lens[b] + s. For every head vector
 * x [D] of k (gamma_k) and, where q is given, of q (gamma_q):
 *   y = x / sqrt(mean_d(x_d^2) + eps) * gamma    (y = x with qk_norm = 0)
 *   (y_a, y_b) -> (y_a c - y_b s, y_a s + y_b c), c = rope_cos[t][i],
 *       s = rope_sin[t][i], (a, b) the i-th pair of rope_layout
 * in fp32, rounded once: q to bf16 into q_out, k to bf16 into k_cache, or with
 * SA_CACHE_FP8 to the e4m3 code nearest to the fp32 quotient y / k_scale[h] (ties
 * to even, |code| at most 448, NaN stays NaN). v goes into v_cache as it is, or as
 * the code of v / v_scale[h].
 * k_sum of the page (where given) gains y before it is rounded; a page's first
 * slot starts its sum anew.
 * Taking tokens back (a guess that was rejected) is setting the length back, but
 * k_sum has gained their keys. sa_cache_accept puts that right for drafted tokens;
 * without it, before more is appended, the sums of the page that
 * the sequence then ends in (page_table[b][n / 64], where n % 64 > 0), [H_kv, D]
 * floats, have to be put back as they were at that length. Those of the pages
 * behind it start anew.
 * Tokens that find no place (t >= 64 max_pages, or t >= rope_rows where tables
 * are given: SA_DEV_CAPACITY; a bad page id: SA_DEV_BAD_CACHE) are left out,
 * with their q_out. The new length does not count the former, which lie behind
 * all others; those of a bad page keep their positions in it, and sa_attn_decode
 * and sa_route_pages leave that page out as well. All else of the caches, k_sum and q_out stays as it was.
 *
 * k, v         device bf16 [B, S, H_kv, D].
 * q, q_out     device bf16 [B, S, H, D] (q_stride; o_stride), or both NULL.
 *              q_out may be q itself with equal strides, else no overlap.
 * gamma_q,     device fp32 [D], 16-byte aligned, or NULL for all ones (and
 * gamma_k      NULL without qk_norm).
 * rope_cos,    device fp32 [rope_rows][D/2], 16-byte aligned; both NULL for
 * rope_sin     no rotation.
 * k_scale,     device fp32 [H_kv], > 0 with a finite reciprocal, or NULL for ones
 * v_scale      (and NULL with SA_CACHE_BF16).
 * seq_lens     the lengths before the call; not modified.
 * new_lens     device int32 [B] in [0, S] (clamped into it), or NULL.
 * lens_out     device int32 [B], or NULL: seq_lens[b] + n_b, at most 64 max_pages
 *              and, where tables are given, max(seq_lens[b], rope_rows); no overlap
 *              with seq_lens or new_lens.
 * Errors: SA_ERR_INVALID_ARG / SA_ERR_UNSUPPORTED before launch; SA_ERR_CUDA.
 */
sa_status sa_cache_append(const sa_cache_params* p, const void* k, const void* v,
                          const void* q, void* q_out, const float* gamma_q,
                          const float* gamma_k, const float* rope_cos, const float* rope_sin,
                          void* k_cache, void* v_cache, const float* k_scale,
                          const float* v_scale, float* k_sum, const int32_t* page_table,
                          const int32_t* seq_lens, const int32_t* new_lens, int32_t* lens_out,
                          int32_t* dev_status, void* stream);

/*
 * sa_cache_append_axes -- sa_cache_append with positions on several axes: a token
 * turns pair i by rope_cos, rope_sin[positions[b][s][axis_of[i]]][i] (fp32
 * [axes->rows][D/2], both given) and is still stored behind its sequence's tokens.
 * So the positions of an image's tokens, or of drafted tokens that lie side by side
 * in a tree, need not follow their slots. No token is left out for its position:
 * lens_out is seq_lens[b] + n_b, at most 64 max_pages. p->rope_rows is not read.
 * positions need only hold the tokens that new_lens counts.
 */
sa_status sa_cache_append_axes(const sa_cache_params* p, const void* k, const void* v,
                               const void* q, void* q_out, const float* gamma_q,
                               const float* gamma_k, const float* rope_cos,
                               const float* rope_sin, const sa_rope_axes* axes, void* k_cache,
                               void* v_cache, const float* k_scale, const float* v_scale,
                               float* k_sum, const int32_t* page_table, const int32_t* seq_lens,
                               const int32_t* new_lens, int32_t* lens_out, int32_t* dev_status,
                               void* stream);

/* Most entries sa_route_pages can list, B*H_kv*min(max_pages, max(page_budget,
 * ceil(P/64) + 1)) (0 on bad params). */
int64_t sa_route_pages_max_nnz(const sa_cache_params* p);

/* Bytes of device workspace sa_route_pages needs (0 on bad params). */
size_t sa_route_pages_workspace_bytes(const sa_cache_params* p);

/*
 * sa_route_pages -- the pages one new token of each sequence attends, per
 * key-value head: the router for a query that is a single token. With
 * n = seq_lens[b] and Nb = ceil(n / 64), page j < Nb of row (b, g) scores
 *   s_j = max over the query heads h of g of  q_h . k_sum[page_table[b][j]][g].
 * Kept are the pages that sa_route always keeps (j < ceil(min(P, n) / 64), and
 * the newest page Nb - 1) and, while fewer than page_budget are, the others by
 * s_j descending (equal s_j: lower j first). Pages that compete are full, so
 * their sums rank as their means do. A head whose score is not a number is
 * passed over; a page without any other head ranks last, as does one with a bad
 * id. (A budget bounds the attention's cost per
 * token; sa_route's threshold does not.) Scores are computed in fp32 with an
 * error bound; those the bound leaves undecided again, to 2^-37 of
 * |q|_1 max |k_sum|, and what that leaves undecided (or fp32 would overflow on)
 * in fp64, so the choice equals that of fp64 scores.
 *
 * q          device bf16 [B, 1, H, D], rotated as the cached keys are.
 * row_ptr    device int32 [B*H_kv + 1]; row r = b*H_kv + g.
 * col_idx    device int32 [col_cap]: page places j, ascending in each row, as
 *            sa_route lists key blocks. Entries beyond col_cap are dropped and
 *            SA_DEV_CAPACITY is raised; sa_route_pages_max_nnz(p) is enough.
 * workspace  device scratch of sa_route_pages_workspace_bytes(p) bytes,
 *            256-byte aligned; its contents on entry do not matter.
 * Errors: as sa_route. max_pages must be <= 2^20, B*H_kv*max_pages and the
 * most entries < 2^31 (SA_ERR_UNSUPPORTED).
 */
sa_status sa_route_pages(const sa_cache_params* p, const void* q, const float* k_sum,
                         const int32_t* page_table, const int32_t* seq_lens, int32_t* row_ptr,
                         int32_t* col_idx, int64_t col_cap, void* workspace, size_t ws_bytes,
                         int32_t* dev_status, void* stream);

/* Bytes of device workspace sa_attn_decode needs (0 on bad params). */
size_t sa_attn_decode_workspace_bytes(const sa_cache_params* p);

/*
 * sa_attn_decode -- attention of one new token per sequence over its cached
 * keys: for head h of sequence b, g = h / (H / H_kv), over the tokens
 * u < seq_lens[b] (the new token's own key among them, once appended)
 *   l_u = softmax_scale * q_h . k_u,   a_u = exp(l_u - max l) / sum exp(.),
 *   o_h = sum_u a_u v_u,               lse_h = max l + log sum exp(l - max l)
 * with k_u, v_u as stored (code * scale). With a route (row_ptr and col_idx)
 * only tokens in the pages listed for row b*H_kv + g. Nothing to attend gives
 * o = 0 and lse = -inf. Whatever lies in the slots behind a sequence's last
 * token, NaN included, has no effect.
 *
 * Precision: exact products with fp32 accumulation and an fp32 softmax; P.V
 * takes P to 2^-21 of itself, as three bf16 terms (with SA_CACHE_FP8 to 2^-21
 * of itself or 2^-40 of the largest, as two fp16 terms, against V in fp16,
 * which holds every e4m3 value) with fp32 accumulation; o is rounded once to bf16. The sums' order, and so the last
 * bit, depends on the lengths in the batch, not on timing.
 *
 * q          device bf16 [B, 1, H, D], rotated as the cached keys are.
 * row_ptr,   device int32 CSR as sa_route_pages writes it, or both NULL for
 * col_idx    every page. One that breaks the contract raises SA_DEV_BAD_ROUTE:
 *            a row whose span does not lie inside [0, col_cap] or that is
 *            longer than max_pages is left out whole; an entry outside
 *            [0, ceil(seq_lens[b] / 64)) or not above the one before it in
 *            its row is left out. col_cap: the entries col_idx holds.
 * k_scale,   as sa_cache_append.
 * v_scale
 * o          device bf16 [B, 1, H, D] (o_stride); no overlap with q.
 * lse        device fp32 [B, H, 1] (natural log), or NULL.
 * workspace  device scratch of sa_attn_decode_workspace_bytes(p) bytes,
 *            256-byte aligned; its contents on entry do not matter.
 * Errors: as sa_attn_sparse; S must be 1 and B*H_kv*max_pages (times
 * ceil(G / 64), G = H / H_kv) < 2^31 (SA_ERR_UNSUPPORTED).
 */
sa_status sa_attn_decode(const sa_cache_params* p, const void* q, const void* k_cache,
                         const void* v_cache, const float* k_scale, const float* v_scale,
                         const int32_t* page_table, const int32_t* seq_lens,
                         const int32_t* row_ptr, const int32_t* col_idx, int64_t col_cap,
                         void* o, float* lse, void* workspace, size_t ws_bytes,
                         int32_t* dev_status, void* stream);

/* ------------------------------------------------------------------------
 * Drafted tokens: a few new tokens of each sequence, appended with sa_cache_append
 * or sa_cache_append_axes, attended all at once, and those of the path that turned
 * out right kept. The calls take the lengths from before the append (seq_lens) and
 * the new tokens' numbers (new_lens), as sa_cache_append does.
 * ---------------------------------------------------------------------- */

/* Most new tokens of a sequence. */
#define SA_TREE_MAX 64

/* Bytes of device workspace sa_attn_tree needs (0 on bad params). */
size_t sa_attn_tree_workspace_bytes(const sa_cache_params* p);

/*
 * sa_attn_tree -- attention of the new tokens of each sequence, a tree (or
 * several) of drafted ones, over its cached keys: new token s < n_b of sequence b
 * (n_b = new_lens[b], S where new_lens is NULL), which lies at position
 * seq_lens[b] + s, sees the tokens u < seq_lens[b] and those new ones that it
 * continues: itself, parents[b][s], that one's parent, and so on to one whose
 * parent is -1. Else as sa_attn_decode, for head h of g = h / (H / H_kv):
 *   l_u = softmax_scale * q_sh . k_u,  a_u = exp(l_u - max l) / sum exp(.),
 *   o_sh = sum_u a_u v_u,              lse_sh = max l + log sum exp(l - max l)
 * With a route (row_ptr, col_idx) only tokens in the pages listed for row
 * b*H_kv + g, and in all pages that hold new tokens, listed or not. What a token
 * does not see has no effect on it, infinities and NaN included.
 * A token without a place (position >= 64 max_pages, SA_DEV_CAPACITY) is left
 * out; rows of o and lse of tokens that are left out or not counted by n_b stay
 * as they were. Tokens whose every page has a bad id get o = 0, lse = -inf.
 *
 * Precision: as sa_attn_decode; where more than 16 rows (new tokens times H / H_kv)
 * share a key-value head, P.V takes P to 2^-16 of itself, as two bf16 terms (with
 * SA_CACHE_FP8 to 2^-21 of itself or 2^-30 of the largest, as two fp16 terms), and
 * with SA_CACHE_FP8 q is taken in fp16 scaled by a power of two for each row, exact but
 * for bits below 2^-39 of its largest element. Long sums in the tensor cores' fp32
 * accumulators are cut, not rounded: over 112,640 tokens o comes out smaller, by about
 * 1.2e-4 of itself (half a bf16 step is up to 39e-4).
 *
 * q          device bf16 [B, S, H, D], rotated as the cached keys are; S at most
 *            SA_TREE_MAX.
 * seq_lens   lengths before the new tokens.
 * parents    device int32: token s of sequence b has parents[b*parent_stride + s]
 *            in [-1, s) (0: one tree for all), or NULL: each continues the one
 *            before it. A parent outside that range counts as -1 and raises
 *            SA_DEV_BAD_TREE.
 * row_ptr,   as sa_attn_decode; entries from seq_lens[b] / 64 on are passed over
 * col_idx    (those pages are attended anyway). sa_route_pages makes one for all
 *            tokens of a sequence from one token's queries and seq_lens.
 * o          device bf16 [B, S, H, D] (o_stride); no overlap with q.
 * lse        device fp32 [B, H, S] (natural log), or NULL.
 * workspace  device scratch of sa_attn_tree_workspace_bytes(p) bytes, 256-byte
 *            aligned; its contents on entry do not matter.
 * Errors: as sa_attn_decode; S above SA_TREE_MAX: SA_ERR_UNSUPPORTED.
 */
sa_status sa_attn_tree(const sa_cache_params* p, const void* q, const void* k_cache,
                       const void* v_cache, const float* k_scale, const float* v_scale,
                       const int32_t* page_table, const int32_t* seq_lens,
                       const int32_t* new_lens, const int32_t* parents, int64_t parent_stride,
                       const int32_t* row_ptr, const int32_t* col_idx, int64_t col_cap, void* o,
                       float* lse, void* workspace, size_t ws_bytes, int32_t* dev_status,
                       void* stream);

/*
 * sa_cache_accept -- the new tokens of the path that turned out right move
 * together: token path[b][i] of sequence b, i < m_b = path_lens[b], from position
 * seq_lens[b] + path[b][i] to seq_lens[b] + i, keys and values. The sequence then
 * ends at seq_lens[b] + m_b; what lies behind that is stale.
 * k_sum (where given) of the pages from seq_lens[b] / 64 to the one that holds the
 * new last token becomes the sum of their keys as they are stored (code * k_scale)
 * up to the new length: with m_b = 0 this takes all new tokens back.
 * A path has to ascend, path[b][i-1] < path[b][i] < SA_TREE_MAX, and to lie in
 * the page table; it counts as far as it does, and SA_DEV_BAD_TREE is raised
 * where it does not. A token whose old or new page has a bad id is not moved
 * (SA_DEV_BAD_CACHE) but counted.
 * The pages that new tokens lie in must belong to one sequence alone.
 *
 * path       device int32: path[b*path_stride + i], i < p->S (at most
 *            SA_TREE_MAX).
 * path_lens  device int32 [B] in [0, S] (clamped into it).
 * lens_out   device int32 [B], or NULL: the new lengths; no overlap with
 *            seq_lens or path_lens.
 * k_scale    as sa_cache_append (read for k_sum only).
 * Errors: SA_ERR_INVALID_ARG / SA_ERR_UNSUPPORTED before launch; SA_ERR_CUDA.
 */
sa_status sa_cache_accept(const sa_cache_params* p, void* k_cache, void* v_cache,
                          const float* k_scale, float* k_sum, const int32_t* page_table,
                          const int32_t* seq_lens, const int32_t* path, int64_t path_stride,
                          const int32_t* path_lens, int32_t* lens_out, int32_t* dev_status,
                          void* stream);

/* ------------------------------------------------------------------------
 * Pages of the pool: who holds them. A page table and an array of reference
 * counts serve the caches of all layers; these calls change only those and name
 * the pages whose contents have to be copied, which sa_cache_copy does a layer at a
 * time. A new table stands for what it says once that is done in every layer, with the
 * key sums where pages are routed: before the next sa_pages_fork or sa_pages_compact,
 * and before tokens are appended or attended.
 *   refs        int32 [n_pages]: how many places hold the page; 0: it is free.
 *               A caller may hold pages of its own (a shared prompt) by counting
 *               them in.
 *   page_table  int32 [B][table_stride]: -1 where a sequence has no page. An entry
 *               outside [-1, n_pages) counts as -1 and raises SA_DEV_BAD_CACHE.
 * A page that is not full belongs to one sequence; full ones may be shared, as
 * nothing is appended to them (so a sequence is not set back into a page that others hold). Free pages are taken in ascending order of their ids,
 * as they are free when the call begins. The workspace serves any of the three.
 * ---------------------------------------------------------------------- */

/* Bytes of device workspace the sa_pages_* calls need for a pool of n_pages and
 * tables of at most `rows` sequences (0 on bad sizes). */
size_t sa_pages_workspace_bytes(int32_t n_pages, int32_t rows);

/*
 * sa_pages_fork -- a new table whose sequence i continues sequence src[i] of the
 * old one (src[i] = -1: an empty one), for beams, several answers to one prompt,
 * reordering and dropping sequences. The first i that continues a sequence takes
 * over its row; every other one shares the full pages, gets a free page in place of
 * one that is not full (its copy), and none behind that. The old table is given up:
 *   refs_out = refs - (places in the old table) + (places in the new one).
 * Where no page is free (SA_DEV_CAPACITY) a sequence keeps its full pages and their
 * tokens only. src[i] outside [-1, B) counts as -1 and raises SA_DEV_BAD_TREE;
 * a seq_lens[b] outside [0, 64 max_pages] counts as the nearest (SA_DEV_BAD_CACHE).
 *
 * page_table, seq_lens, refs   the old state; not modified (but refs_out may be refs).
 * src         device int32 [N].
 * table_out   device int32 [N][out_stride], max_pages entries a row; no overlap
 *             with page_table.
 * lens_out    device int32 [N]; no overlap with seq_lens.
 * refs_out    device int32 [n_pages]: refs itself, or no overlap with it.
 * moves       device int32 [N][2]: (page, its copy), n_moves[0] of them, in the
 *             order of i.
 * n_moves     device int32 [1].
 * workspace   device scratch of sa_pages_workspace_bytes(n_pages, max(B, N))
 *             bytes, 256-byte aligned.
 * Errors: SA_ERR_INVALID_ARG / SA_ERR_UNSUPPORTED (B or N above 16,384, n_pages or
 * max_pages from 2^25 on) / SA_ERR_CAPACITY before launch; SA_ERR_CUDA.
 */
sa_status sa_pages_fork(int32_t n_pages, int32_t max_pages, int32_t B, int32_t N,
                        const int32_t* page_table, int64_t table_stride,
                        const int32_t* seq_lens, const int32_t* refs, const int32_t* src,
                        int32_t* table_out, int64_t out_stride, int32_t* lens_out,
                        int32_t* refs_out, int32_t* moves, int32_t* n_moves, void* workspace,
                        size_t ws_bytes, int32_t* dev_status, void* stream);

/*
 * sa_pages_resize -- every sequence holds exactly the pages for seq_lens[b] +
 * more_lens[b] tokens (+ more where more_lens is NULL), in place: places before that
 * without a page get a free one, row by row, pages behind it are given back. Where no
 * page is free, or beyond max_pages, SA_DEV_CAPACITY is raised and places stay empty.
 * seq_lens = 0 with more = 0 frees a sequence. The wanted length counts as at
 * least 0 (SA_DEV_BAD_CACHE where it is below).
 */
sa_status sa_pages_resize(int32_t n_pages, int32_t max_pages, int32_t B, int32_t* page_table,
                          int64_t table_stride, int32_t* refs, const int32_t* seq_lens,
                          const int32_t* more_lens, int32_t more, void* workspace,
                          size_t ws_bytes, int32_t* dev_status, void* stream);

/*
 * sa_pages_compact -- the pages in use move to the front of the pool: with n_used
 * pages in use (refs > 0), the k-th of those at or behind n_used takes the place of
 * the k-th free one before it. Afterwards pages [0, n_used) are in use, so the pool
 * behind them can be given back or a checkpoint written without holes.
 *
 * table_out   device int32 [B][out_stride]: page_table with the new ids; page_table
 *             itself (with the same stride), or no overlap.
 * refs_out    refs itself, or no overlap.
 * moves       device int32 [n_pages / 2][2] (at least one): (page, its new id),
 *             ascending, n_moves[0] of them. new ids and old ones are distinct.
 * n_used      device int32 [1].
 * B may be 0 (page_table, table_out NULL): refs alone.
 */
sa_status sa_pages_compact(int32_t n_pages, int32_t max_pages, int32_t B,
                           const int32_t* page_table, int64_t table_stride, const int32_t* refs,
                           int32_t* table_out, int64_t out_stride, int32_t* refs_out,
                           int32_t* moves, int32_t* n_moves, int32_t* n_used, void* workspace,
                           size_t ws_bytes, int32_t* dev_status, void* stream);

/*
 * sa_cache_copy -- the keys, values and key sums (k_sum, where given) of page
 * moves[i][0] to page moves[i][1], i < n_moves[0] (at most move_cap; all of them
 * where n_moves is NULL). No page may be written twice or both read and written. A
 * pair with an id outside [0, n_pages) is left out (SA_DEV_BAD_CACHE). p: H_kv, D,
 * n_pages, cache_format and the caches' strides are read.
 */
sa_status sa_cache_copy(const sa_cache_params* p, void* k_cache, void* v_cache, float* k_sum,
                        const int32_t* moves, int64_t move_cap, const int32_t* n_moves,
                        int32_t* dev_status, void* stream);

/* Decodes *dev_status bits into the most severe sa_status (SA_OK if 0). */
sa_status sa_dev_status_decode(int32_t dev_status);

/* A static, NUL-terminated name of the status. */
const char* sa_status_string(sa_status s);

#ifdef __cplusplus
}
#endif

#endif /* SA_GB300_H */
