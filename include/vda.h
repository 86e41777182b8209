/*
 * vda.h - C ABI of the B200 (sm_100a) bidirectional Video Delta Attention branch.
 *
 * Paper: "Video DeltaNet: A Video-Native Hybrid Attention for Livestream Video
 * Generation" (arXiv 2609.20744).  The library computes the linear branch of
 * one hybrid attention block (Algorithm 1, steps 3-7; shown here with the
 * decay gate fixed to 1, see "Decay" below for the general form):
 *
 *   for every batch b, head h and interior latent frame t:
 *     A_t = K_t^T Diag(beta_t) K_t,  B_t = V_t^T Diag(beta_t) K_t     (Eq. 3b)
 *     forward scan  P_t = (P_{t-1} + B_t)(I + A_t)^{-1}, P_{-1} = S0_fwd (Eq. 5)
 *     reverse scan  R_t = (R_{t+1} + B_t)(I + A_t)^{-1}, R_T  = S0_rev
 *     query chunk c reads  S~_c = P_{l-1} + R_{h+1}  just outside its local
 *     window [l, h] (Appendix A.3, Eq. A.4; a side without distant frames reads
 *     its initial state), o = S~_c q                                   (Eq. 1a)
 *     out = sigmoid(gate) * w * o / sqrt(mean_{d_v}(o^2) + eps)        (Eq. 1c)
 *
 * Conventions shared by every entry point
 *   - Layouts are contiguous and row-major:
 *       q, k      [B, H, T, U, d_k]      v, gate, out  [B, H, T, U, d_v]
 *       beta      [B, H, T, U]  float32 (write gates, >= 0)
 *       rms_weight[d_v]         float32, shared by all heads
 *       S0_fwd, S0_rev [B, H, d_v, d_k] float32; the state maps keys to
 *                 values, o = S q.  NULL means the zero state.
 *     T counts interior frames only: the caller has already removed the two
 *     boundary anchor frames (Algorithm 1, step 2).
 *   - Chunks tile the interior frame index from 0: chunk c holds frames
 *     [c*chunk, (c+1)*chunk); the last chunk may be shorter.  The local window
 *     of chunk c is chunks c-window_chunks .. c+window_chunks clipped to the
 *     clip; a window covering the whole clip yields
 *     RMSNorm((S0_fwd + S0_rev) q) * sigmoid(gate), which is 0 for zero S0.
 *   - bf16 tensors are passed as uint16_t bit patterns (IEEE bfloat16).
 *   - All pointers except those documented as host pointers are device
 *     pointers owned by the caller; the library never frees them and keeps no
 *     reference after the call returns.  Device pointers must be 16-byte
 *     aligned.
 *   - Work is enqueued on `stream` (a cudaStream_t passed as void*; NULL is
 *     the legacy default stream) and the call returns without synchronising,
 *     except where stated.
 *   - Decay (Eq. 2 and Appendix A.3, Eq. A.4): with vda_args.alpha set, both
 *     scans decay the entering state channel-wise before each frame update,
 *       P_t = (P_{t-1} Diag(alpha_t) + B_t)(I + A_t)^{-1}   (and R_t alike,
 *       with the frame's own alpha_t),
 *     and query frame t reads the bridged states
 *       S~_t = P_{l-1} Diag(prod_{r=l..t} alpha_r) + R_{h+1} Diag(prod_{r=t..h} alpha_r)
 *     (a side without distant frames bridges its initial state).  alpha is
 *     [B, H, T, d_k] float32 with values in [0, 1].  vda_forward and
 *     vda_forward_f32 have no decay (alpha = 1); vda_forward_ex,
 *     vda_forward_host and vda_forward_noalloc take it from vda_args.
 *   - Supported sizes: d_k == d_v in {16, 32, 64, 128}; chunk >= 1;
 *     window_chunks >= 0; B, H, T, U >= 1.  d = 128 and d = 64 with bf16 I/O
 *     run on the tcgen05 tensor-core kernels (at d = 64 with the FP32
 *     Gauss-Jordan inverse); the other sizes run on SIMT kernels.
 *   - Errors: every argument is validated before any launch; no exception
 *     crosses the ABI.  See vda_status.
 */
#ifndef VDA_H
#define VDA_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define VDA_API __attribute__((visibility("default")))
#else
#define VDA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum vda_status {
  VDA_OK = 0,
  VDA_ERR_INVALID_ARGUMENT = 1, /* NULL required pointer, size <= 0, misaligned pointer */
  VDA_ERR_UNSUPPORTED = 2,      /* valid but unsupported sizes (d_k != d_v, d not in the list) */
  VDA_ERR_WORKSPACE = 3,        /* caller workspace smaller than vda_workspace_bytes() */
  VDA_ERR_CUDA = 4,             /* a CUDA runtime call or kernel launch failed */
  VDA_ERR_TIMEOUT = 5           /* a kernel gave up waiting on a barrier (see vda_device_status) */
} vda_status;

typedef enum vda_dtype {
  VDA_BF16 = 0, /* q, k, v, gate, out (and text tokens) are bfloat16 */
  VDA_F32 = 1   /* ... are float32 */
} vda_dtype;

/* How the forward and reverse scans of Section 2.2 run on the tensor-core
 * path at d = 128 (bf16); the other paths always scan frame by frame.  Both give
 * the same boundary states up to rounding.
 *   VDA_SCAN_FRAMES: one sequential chain of T frame updates per (b, h,
 *     direction), S <- (S Diag(alpha_t) + B_t) M_t.
 *   VDA_SCAN_CHUNKS: the chunk-wise scan of Section 5 ("Chunk-wise scans",
 *     Appendix A.1): every chunk's frames are first composed, in parallel,
 *     into one affine map S -> S P_c + J_c, then each chain runs its NC maps.
 *     About twice the tensor-core work on a chain of chunk + NC steps; it pays
 *     when few (b, h) pairs share the GPU.
 *   VDA_SCAN_AUTO: the library picks by the number of (b, h) pairs.
 * VDA_SCAN_CHUNKS with more than 2^31 - 1 composition CTAs (4 B H NC) returns
 * VDA_ERR_UNSUPPORTED. */
typedef enum vda_scan_form {
  VDA_SCAN_AUTO = 0,
  VDA_SCAN_FRAMES = 1,
  VDA_SCAN_CHUNKS = 2
} vda_scan_form;

/* Full argument block of vda_forward_ex. */
typedef struct vda_args {
  int dtype;                  /* vda_dtype of q, k, v, gate, out */
  const void* q;              /* [B,H,T,U,d_k] */
  const void* k;              /* [B,H,T,U,d_k] */
  const void* v;              /* [B,H,T,U,d_v] */
  const float* beta;          /* [B,H,T,U] */
  const void* gate;           /* [B,H,T,U,d_v] sigmoid-gate logits */
  const float* rms_weight;    /* [d_v] */
  const float* S0_fwd;        /* [B,H,d_v,d_k] or NULL */
  const float* S0_rev;        /* [B,H,d_v,d_k] or NULL */
  void* out;                  /* [B,H,T,U,d_v] */
  int B, H, T, U, d_k, d_v;
  int chunk;                  /* frames per chunk (the paper: 5) */
  int window_chunks;          /* window radius in chunks (the paper: 1) */
  float eps;                  /* RMSNorm epsilon; <= 0 selects 1e-6 */
  void* stream;               /* cudaStream_t */
  const float* alpha;         /* [B,H,T,d_k] decay gates in [0,1] (Eq. 2), or NULL: no decay */
  int scan_form;              /* vda_scan_form; 0 (zero-initialised args) = VDA_SCAN_AUTO */
} vda_args;

/* Bidirectional VDA forward, bf16 I/O.  Takes its workspace stream-ordered
 * (cudaMallocAsync / cudaFreeAsync on `stream`).  Returns vda_status. */
VDA_API int vda_forward(const uint16_t* q, const uint16_t* k, const uint16_t* v,
                const float* beta, const uint16_t* gate, const float* rms_weight,
                const float* S0_fwd, const float* S0_rev,
                int B, int H, int T, int U, int d_k, int d_v,
                int chunk, int window_chunks, uint16_t* out, void* stream);

/* Same as vda_forward with float32 q, k, v, gate and out. */
VDA_API int vda_forward_f32(const float* q, const float* k, const float* v,
                    const float* beta, const float* gate, const float* rms_weight,
                    const float* S0_fwd, const float* S0_rev,
                    int B, int H, int T, int U, int d_k, int d_v,
                    int chunk, int window_chunks, float* out, void* stream);

/* Bytes of device workspace vda_forward_ex needs for these sizes (0 when the
 * sizes are invalid).  The workspace holds the per-frame statistics and
 * transitions and the chunk-boundary states, all float32. */
VDA_API size_t vda_workspace_bytes(int B, int H, int T, int U, int d_k, int d_v,
                           int chunk, int dtype);

/* Forward with a caller-supplied device workspace (>= vda_workspace_bytes,
 * 256-byte aligned) and optional debug outputs:
 *   states_out [2, B, H, NC+1, d_v, d_k] float32, NC = ceil(T / chunk):
 *     states_out[0,b,h,j] = state after absorbing frames [0, j*chunk) forward
 *                           from S0_fwd (j = 0 is S0_fwd, j = NC the final P);
 *     states_out[1,b,h,j] = state after absorbing frames [j*chunk, T) in
 *                           reverse from S0_rev (j = NC is S0_rev).
 *   stats_out  [3, B, H, T, d, d] float32: A_t, B_t and M_t = (I + A_t)^{-1}.
 * Either may be NULL.  Resuming: passing states_out[0,b,h,NC] of one call as
 * S0_fwd of a call on the following frames continues the forward scan. */
VDA_API int vda_forward_ex(const vda_args* args, void* workspace, size_t workspace_bytes,
                   float* states_out, float* stats_out);

/* Text state of Eq. (1b) for one prompt per (b, h): one frame-wise update of
 * the zero state with the L prompt tokens treated as one frame,
 *   S_out = B'(I + A')^{-1},  A' = K'^T Diag(beta') K',  B' = V'^T Diag(beta') K'.
 * k_text [B,H,L,d_k], v_text [B,H,L,d_v] (dtype), beta_text [B,H,L] float32
 * (pass the halved gates to obtain S_T/2 for both scans), S_out [B,H,d_v,d_k]
 * float32.  Workspace: vda_text_state_workspace_bytes(), device, 256-byte
 * aligned. */
VDA_API size_t vda_text_state_workspace_bytes(int B, int H, int L, int d_k, int d_v, int dtype);
VDA_API int vda_text_state(int dtype, const void* k_text, const void* v_text, const float* beta_text,
                   int B, int H, int L, int d_k, int d_v, float* S_out,
                   void* workspace, size_t workspace_bytes, void* stream);

/* End-to-end forward from HOST buffers: every array of `args` (q, k, v, beta,
 * gate, rms_weight, S0_fwd, S0_rev, out) is a host pointer (page-locked for
 * overlap); the call copies the inputs to the device, runs the forward and
 * copies `out` back, pipelining groups of heads over two streams (copy and
 * compute) so that transfers overlap the kernels.  Every group takes the
 * scan form the whole problem takes, so `out` equals vda_forward_ex's bit for
 * bit.  `device_buffer` is caller device memory of at least
 * vda_forward_host_bytes() bytes (256-byte aligned).  Synchronous: returns
 * when `out` is complete on the host. */
VDA_API size_t vda_forward_host_bytes(int B, int H, int T, int U, int d_k, int d_v,
                              int chunk, int dtype);
VDA_API int vda_forward_host(const vda_args* host_args, void* device_buffer, size_t device_bytes);

/* Forward without any allocation, for callers that cannot allocate device
 * memory: host frameworks that own all device memory through their own
 * allocator and have no way to hand this library a workspace, plugins loaded
 * into such hosts, and fixed-footprint serving or real-time loops whose
 * policy forbids allocator calls once they are running (a cudaMalloc there
 * can block, fail under memory pressure, or synchronise the device).  Same
 * arguments and result as vda_forward_ex with no workspace and no debug
 * outputs; the scratch (statistics, transitions and chunk-boundary states)
 * lives in one fixed array of VDA_NOALLOC_SCRATCH_BYTES inside the library,
 * which every GPU that loads the library holds until the process exits.
 *   - Returns VDA_ERR_WORKSPACE when the sizes need more scratch than that
 *     (vda_workspace_bytes() > VDA_NOALLOC_SCRATCH_BYTES); nothing is launched.
 *   - Every call looks up the array's device address in the current context
 *     with the CUDA runtime (cudaGetSymbolAddress; no allocation), so the
 *     address is never stale after cudaDeviceReset or under another context.
 *     The first lookup in a context may load the library's device code; make
 *     the first call on each device before any stream capture begins.
 *   - Calls share the one array: two calls whose work overlaps on the GPU
 *     (different streams, or different host threads, without ordering between
 *     them) race and corrupt each other's results.  Every scratch word is
 *     written before it is read in each call, so nothing left by an earlier
 *     call leaks into a later one.
 * The paper has no counterpart to this entry point; it is a deployment aid. */
#define VDA_NOALLOC_SCRATCH_BYTES ((size_t)16 << 20)
VDA_API int vda_forward_noalloc(const vda_args* args);

/* Synchronises `stream`, then reads and clears the library's device error
 * word for the current device: returns VDA_ERR_TIMEOUT if a kernel gave up a
 * bounded wait since the last call, VDA_ERR_CUDA on a CUDA error, else VDA_OK. */
VDA_API int vda_device_status(void* stream);

/* Failure-detection self test: launches one kernel that waits, with a bounded
 * poll, on a device flag that nothing sets.  After max_polls polls (1 ..
 * 1000000, about 0.1 us each) it gives up, records a wait time-out in the
 * device error word and returns normally, so the context stays usable; the
 * next vda_device_status(stream) returns VDA_ERR_TIMEOUT and clears it.
 * No compute path calls this; it exists to test failure detection without
 * a GPU fault.  Returns vda_status. */
VDA_API int vda_selftest_wait_timeout(int max_polls, void* stream);

/* Per-stage device timing for profiling.  vda_timing_enable(n) makes the next
 * n forward calls record a CUDA event just before and just after each kernel
 * launch, on the launch's stream; vda_timing_read(ms, 4, &calls) synchronises
 * on the recorded events and writes, per stage (stats, inverse, scan,
 * readout), the milliseconds summed over that stage's launches and calls, and
 * the number of calls recorded, then disables timing and releases the events.
 * vda_timing_enable(0) disables it. */
VDA_API int vda_timing_enable(int max_calls);
VDA_API int vda_timing_read(float* stage_ms, int n_stages, int* calls);

/* Number of kernel launches one vda_forward_ex call with these sizes makes
 * without a decay gate and with scan_form VDA_SCAN_AUTO on the current device
 * (the chunk-wise scans take two launches); with vda_args.alpha set the call
 * makes one more (the bridge products of Eq. A.4). */
VDA_API int vda_launches_per_forward(int B, int H, int T, int U, int d_k, int d_v, int chunk, int dtype);

/* ---------------------------------------------------------------------------
 * Feature preparation of the linear branch (Section 2.3; the fused "VDA-Prep"
 * step of Section 5), the step ahead of vda_forward:
 *   q' = L2(q),  k' = L2(SiLU(conv(k))),  v' = SiLU(conv(v))
 * conv = a depthwise 5 x 5 spatial filter over the Hl x Wl latent grid then a
 * depthwise five-tap temporal filter over the interior frames, both
 * cross-correlations with zero padding 2 on every side; L2(x) =
 * x / sqrt(sum(x^2) + eps) over the head dimension.
 *   q_in, k_in, v_in  [B, T, U, H, d] bf16 (the projections of the interior
 *                     video tokens, heads inner; token u = y * Wl + x)
 *   wk_s, wv_s        [H, d, 5, 5] float32, wk_t, wv_t [H, d, 5] float32
 *   q_out, k_out, v_out [B, H, T, U, d] bf16 (the layout vda_forward reads)
 * Supported: bf16, d in {16, 32, 64, 128}, at most 8 grid columns per
 * thread slice (Wl <= 8 * 1024 / d) and the staged rows, the spatial taps and
 * one fp32 output row (about 5 (Wl + 4) * 2 d + 100 d + 4 d Wl bytes) within
 * the device's shared memory (Wl <= 64 at d = 128).  Inputs and outputs must
 * not overlap.
 * Returns vda_status. */
typedef struct vda_prep_args {
  const void* q_in;
  const void* k_in;
  const void* v_in;
  const float* wk_s;
  const float* wk_t;
  const float* wv_s;
  const float* wv_t;
  void* q_out;
  void* k_out;
  void* v_out;
  int B, H, T, Hl, Wl, d;
  float eps;                  /* L2 epsilon; <= 0 selects 1e-6 */
  void* stream;               /* cudaStream_t */
} vda_prep_args;

VDA_API int vda_prep(const vda_prep_args* args);

/* ---------------------------------------------------------------------------
 * The Softmax branch of the hybrid block (Section 2.1 and the fused QK-norm +
 * RoPE of Section 5): the norm and rotation of queries and keys, which may
 * append K and V to a paged cache, and the attention that reads the cache.
 *
 * Rows of a tensor [N tokens, heads, d]: channel 0 of (token, head) lies at
 * data + token * token_stride + head * head_stride (in elements, both >= 0),
 * the d channels are contiguous.  data is 16-byte aligned and the strides are
 * multiples of 16 bytes, so slices of a joint [q | k | v] projection and
 * head-major tensors are taken as they are.  Inputs may have stride 0
 * (broadcast); rows of outputs must not overlap, neither one another nor an
 * input: there is no form in place.  Such a call is refused where the larger
 * strides of the two are alike, as those of views of one tensor are, or one is
 * contiguous; other overlaps are not looked for. */
typedef struct vda_rows {
  void* data;
  int64_t token_stride;
  int64_t head_stride;
} vda_rows;

/* For every token and head, with x its d channels and w the tensor's weight:
 *   x^ = x / sqrt(mean(x^2) + eps),  z = w x^,  y = R z
 * R turns pair p of the first rot channels by position[axis[p]] * frequencies[p]:
 *   (y_i, y_j) = (z_i cos - z_j sin, z_j cos + z_i sin),
 *   (i, j) = (p, p + rot / 2), or (2 p, 2 p + 1) when interleaved.
 * Sums are held in 32 bits or more; the phase of an integer position is off
 * by at most 2^-25 + |position| 2^-64 turns for frequencies of either sign up
 * to 2^40.  y is rounded once.
 * With slots set, k's y and v (unchanged) also go to place slots[token] =
 * page * page_size + offset of the paged cache [pages, Hk, page_size, d]; a
 * token whose slot lies outside [0, pages * page_size) is not stored (give -1
 * for padding), and two tokens must not share a slot.
 * Supported: d in {16, 32, 64, 128}, rot a multiple of 16 in [0, d], axes in
 * 1..8.  N = 0 is a valid empty call.  Returns vda_status. */
typedef struct vda_qk_args {
  int dtype;                  /* vda_dtype of q, k, v and the cache */
  vda_rows q_in;              /* [N, Hq, d] */
  vda_rows k_in;              /* [N, Hk, d] */
  vda_rows v_in;              /* [N, Hk, d], read only when slots is set */
  vda_rows q_out;             /* [N, Hq, d] */
  vda_rows k_out;             /* [N, Hk, d]; data may be NULL when slots is set */
  const float* q_weight;      /* [d] or NULL: ones */
  const float* k_weight;      /* [d] or NULL: ones */
  const int* positions;       /* [N, axes]; NULL when rot = 0 */
  const double* frequencies;  /* [rot / 2] radians per position; NULL when rot = 0 */
  const int* axis;            /* [rot / 2] axis of each pair (outside [0, axes): not turned); NULL when rot = 0 */
  const int64_t* slots;       /* [N] or NULL: no cache */
  void* k_cache;              /* [pages, Hk, page_size, d] */
  void* v_cache;              /* [pages, Hk, page_size, d] */
  int N, Hq, Hk, d;
  int axes, rot, interleaved;
  int pages, page_size;       /* >= 1 when slots is set */
  float eps;                  /* finite; <= 0 selects 1e-6 */
  void* stream;               /* cudaStream_t */
} vda_qk_args;

VDA_API int vda_qk_norm_rope(const vda_qk_args* args);

/* Gradient of vda_qk_norm_rope: from the gradients of q_out and k_out and the
 * forward's inputs, the gradients of q_in and k_in and of the weights,
 *   g = R^T dy,  dw = sum over tokens and heads of g x^,
 *   dx = (g w - x^ mean(g w x^)) / sqrt(mean(x^2) + eps).
 * The norm is computed again from q_in and k_in.  The weight gradients are
 * float32 sums in a fixed order: the same inputs give the same bits.
 * Workspace: vda_qk_grad_workspace_bytes(d), device, 256-byte aligned; it may
 * be NULL when both weight gradients are.  N = 0 sets the weight gradients to
 * zero. */
typedef struct vda_qk_grad_args {
  int dtype;
  vda_rows dq_out;            /* [N, Hq, d] gradient of q_out */
  vda_rows dk_out;            /* [N, Hk, d] gradient of k_out */
  vda_rows q_in;              /* [N, Hq, d] */
  vda_rows k_in;              /* [N, Hk, d] */
  vda_rows dq_in;             /* [N, Hq, d] result */
  vda_rows dk_in;             /* [N, Hk, d] result */
  const float* q_weight;
  const float* k_weight;
  float* dq_weight;           /* [d] result, or NULL */
  float* dk_weight;           /* [d] result, or NULL */
  const int* positions;
  const double* frequencies;
  const int* axis;
  int N, Hq, Hk, d;
  int axes, rot, interleaved;
  float eps;                  /* as in vda_qk_args */
  void* stream;
} vda_qk_grad_args;

VDA_API size_t vda_qk_grad_workspace_bytes(int d);
VDA_API int vda_qk_norm_rope_backward(const vda_qk_grad_args* args, void* workspace, size_t workspace_bytes);

/* Attention of new tokens over a paged cache that already holds their keys
 * and values (vda_qk_norm_rope with slots puts them there).  The n = q_start[b +
 * 1] - q_start[b] new tokens of sequence b are its last n positions: token i
 * stands at position p = kv_len[b] - n + i.  Key j of sequence b lies in page
 * block_table[b][j / page_size] at offset j % page_size.
 *   o = sum_j softmax_j(scale q k_j) v_j,  lse = log sum_j exp(scale q k_j)
 * over the keys j < kv_len[b] that the token sees:
 *   block = 0:  all of them;
 *   block >= 1: positions fall into blocks floor((p - anchors) / block); the
 *               token sees its own block whole (block = 1: causal by token,
 *               block = tokens of a chunk: causal by chunk), the window_blocks
 *               blocks before it (< 0: every block before it) and, of the first
 *               `anchors` keys, those before the end of its own block.  Anchors
 *               are keys that came first: a token among them, or in a block
 *               that ends among them, does not see the later ones.
 * Keys that are no such run, as those of a clip's chunk (the chunks on both
 * sides of it, the anchor frames at both ends): give each chunk as a sequence
 * with block = 0 whose row of the block table lists the pages of what it
 * sees.  Rows may share pages; all but the last page of a row must be full.
 * A token that sees nothing (p < 0, or no key) gets o = 0 and lse = -inf.  A
 * key whose page id lies outside [0, pages) is not seen, whatever mask holds
 * (an evicted page).  What lies in the cache at places that no new token of
 * the sequence sees does not matter, NaN included; a value that is not finite
 * at a key which one token sees can reach the other tokens of the sequence.
 * Query heads h with h / (Hq / Hk) equal share a KV head.  Tokens before
 * q_start[0] and from q_start[B] on are left as they were.
 * q, out, lse: rows as described above (on the tensor cores q is not a
 * broadcast: its strides are at least 16 bytes); lse [N, Hq] float32 contiguous or NULL.
 * S, the softmax's maximum and sum and the output sums are float32; on the
 * tensor cores (bf16, d = 64 or 128, page_size a power of two from 8 on) the
 * weights are rounded to bf16 before their product with
 * V, their sum is not.  Other types and sizes run on a SIMT kernel in float32.
 * Supported: d in {16, 32, 64, 128}; Hq / Hk up to 128 on the tensor cores,
 * 64 elsewhere; pages * Hk < 2^31.  The lengths and the table are read on the
 * device: a captured call follows them.  N = 0 is a valid empty call, with B
 * and max_pages from 0 on and without the arrays of sequences.
 * Workspace: vda_paged_attention_workspace_bytes(), device, 256-byte aligned;
 * calls that may overlap need one each.  Returns vda_status. */
typedef struct vda_attn_args {
  int dtype;                  /* vda_dtype of q, the cache and out */
  vda_rows q;                 /* [N, Hq, d] */
  const void* k_cache;        /* [pages, Hk, page_size, d] */
  const void* v_cache;        /* [pages, Hk, page_size, d] */
  const int* block_table;     /* [B, max_pages], rows table_stride apart */
  const int* kv_len;          /* [B] keys of each sequence, the new tokens' among them */
  const int* q_start;         /* [B + 1] first new token of each sequence, ascending */
  vda_rows out;               /* [N, Hq, d] */
  float* lse;                 /* [N, Hq] or NULL */
  int64_t table_stride;
  int N, B, Hq, Hk, d;
  int pages, page_size, max_pages;
  int block, window_blocks, anchors;
  float scale;                /* > 0; 0 selects 1 / sqrt(d) */
  void* stream;               /* cudaStream_t */
} vda_attn_args;

/* 0 when the sizes are invalid or unsupported. */
VDA_API size_t vda_paged_attention_workspace_bytes(int dtype, int N, int B, int Hq, int Hk, int d, int page_size);
VDA_API int vda_paged_attention(const vda_attn_args* args, void* workspace, size_t workspace_bytes);

/* Human-readable name of a vda_status value. */
VDA_API const char* vda_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* VDA_H */
