/*
 * gdn.h — C ABI of the packed gated-delta-rule (GDN) prefill library for sm_103a.
 *
 * What the library computes
 * -------------------------
 * The gated delta rule (Gated Delta Networks, Yang, Kautz & Hatamizadeh, 2024) is the
 * linear-attention layer of the Qwen3.5/3.6 hybrid models ("hybrid attention architecture
 * used by Qwen3.5-style models", vLLM-Ascend tutorial "Qwen3.6-35B-A3B", §1 Introduction).
 * For every packed prompt n and value head h, with key head hk = h / (H_v / H_k), the
 * state S (d_v x d_k, fp32) evolves token by token:
 *
 *     q_t, k_t <- q_t / ||q_t||, k_t / ||k_t||          (when qk_l2norm != 0)
 *     g_t = exp(a_t)
 *     S_t = g_t S_{t-1} - beta_t (g_t S_{t-1} k_t - v_t) k_t^T
 *     o_t = scale * S_t q_t
 *
 * Many prompts share one pass ("packed passes", sparkinfer v0.6.28 release notes, intro).
 * Each prompt may start from its own initial state (a prefix-cache hit) and the pass emits
 * state snapshots at requested prompt positions ("prefix-cache checkpoint", same release
 * notes, bullets 2-4). A one-token decode update serves sequences that are decoding
 * ("packed GDN decode", vllm.cpp "vLLM, online serving", lever 2b).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Every pointer named *_host is host memory; every other data pointer is device memory
 *    of the current CUDA device, owned by the caller, and must stay valid until the work
 *    queued on `stream` has finished. The library never frees caller memory.
 *  - `stream` is a cudaStream_t passed as void* (NULL = legacy default stream). All
 *    device work is asynchronous on it.
 *  - All arguments are validated on the host before anything is enqueued; on an error
 *    nothing is launched and the status says why ("reject unsupported combinations before
 *    model loading", pegainfer PR #786, Changes). A failed launch returns GDN_ERR_CUDA.
 *  - No call logs, throws or exits.
 *  - Token-major layouts: q, k are [T][H_k][d_k]; v, o are [T][H_v][d_v]; a and beta are
 *    [T][H_v]; states are [.][H_v][d_v][d_k] fp32 with d_k contiguous (row = value dim).
 *    T = cu_seqlens_host[num_seqs]. Device buffers must be 16-byte aligned.
 */
#ifndef GDN_H_
#define GDN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define GDN_ABI_VERSION 1

typedef enum gdn_status {
  GDN_OK = 0,
  GDN_ERR_INVALID_ARGUMENT = 1,   /* malformed sizes, pointers, offsets or positions  */
  GDN_ERR_UNSUPPORTED = 2,        /* well-formed but outside what the kernels cover   */
  GDN_ERR_WORKSPACE_TOO_SMALL = 3,
  GDN_ERR_CUDA = 4,               /* a CUDA runtime call or launch failed             */
  GDN_ERR_DEVICE_TIMEOUT = 5,     /* a bounded device-side wait gave up               */
  GDN_ERR_POOL_EXHAUSTED = 6,     /* pinned snapshot pool range out of bounds         */
  GDN_ERR_BUSY = 7                /* the handle's prefill stream already has a prefill */
} gdn_status;

typedef enum gdn_dtype {
  GDN_F32 = 0,   /* q, k, v, o in fp32 */
  GDN_BF16 = 1   /* q, k, v, o in bf16; a, beta and all states stay fp32 */
} gdn_dtype;

/* How the `a` and `beta` arrays of a call are read. */
typedef enum gdn_gate_mode {
  GDN_GATES_DIRECT = 0,  /* a = log-decay (g = exp(a)), beta = write strength, as given */
  GDN_GATES_RAW = 1      /* raw projections of the Qwen3.5/3.6-style GDN layer, turned into
                            gates in the kernel: a = -exp(A_log[h]) * softplus(a_raw +
                            dt_bias[h]), beta = sigmoid(b_raw) (fp32 arithmetic) */
} gdn_gate_mode;

/* Layer shape and gate inputs. Supported: head_dim_k == head_dim_v in {64, 128},
 * num_v_heads a positive multiple of num_k_heads, chunk_size == 64. With gate_mode ==
 * GDN_GATES_RAW, a_log and dt_bias must be non-NULL device arrays of H_v floats (unused
 * otherwise). */
typedef struct gdn_config {
  int32_t num_k_heads;   /* H_k */
  int32_t num_v_heads;   /* H_v; value head h reads key head h / (H_v / H_k)       */
  int32_t head_dim_k;    /* d_k */
  int32_t head_dim_v;    /* d_v */
  int32_t chunk_size;    /* C: token block of the chunked scan; checkpoint grid     */
  float scale;           /* output scale, usually 1/sqrt(d_k)                       */
  int32_t qk_l2norm;     /* nonzero: q, k <- x / sqrt(x.x + 1e-6) per token and head */
  int32_t io_dtype;      /* gdn_dtype of q, k, v, o                                 */
  int32_t gate_mode;     /* gdn_gate_mode of a and beta                              */
  const float* a_log;    /* [H_v] device fp32 per-head log decay rate (GATES_RAW)    */
  const float* dt_bias;  /* [H_v] device fp32 per-head bias of a_raw (GATES_RAW)     */
} gdn_config;

typedef struct gdn_handle gdn_handle;

/* Library ABI version (GDN_ABI_VERSION of the build). */
int32_t gdn_abi_version(void);

/* Static, NUL-terminated name of a status code; unknown codes give "unknown status". */
const char* gdn_status_string(int32_t status);

/* Create a handle bound to CUDA device `device`. The handle owns a pinned host snapshot
 * pool of `pinned_pool_bytes` (0 = none), allocated here, once, rather than in the middle
 * of a pass (sparkinfer v0.6.28, bullet on pinned host buffers), a side stream for
 * checkpoint copies, a pinned staging ring for work lists, and events. On success *out
 * receives the handle. Errors: INVALID_ARGUMENT (out NULL, device out of range), CUDA. */
gdn_status gdn_handle_create(int32_t device, size_t pinned_pool_bytes, gdn_handle** out);

/* Drain the handle's side stream and staging ring, then free what the handle owns
 * ("drain the prefill stream on error, cancellation, drop, and shutdown", pegainfer PR
 * #786, Changes). NULL is accepted and ignored. */
gdn_status gdn_handle_destroy(gdn_handle* handle);

/* Host address and size of the handle's pinned snapshot pool. */
gdn_status gdn_pool_info(gdn_handle* handle, void** host_ptr, size_t* bytes);

/* Kernel choice for later prefill calls on this handle:
 *   0 = automatic: the tensor-core chunked kernel where it applies (bf16 io, d = 64 or
 *       128; d = 64 heads run zero-padded to 128, exact), in the schedule
 *       gdn_chunked_schedule names for the pack; otherwise (fp32 io) the token-serial
 *       CUDA-core kernel;
 *   1 = always the token-serial kernel (a cross-check path);
 *   2 = the chunked kernel's pipelined schedule, 3 = its throughput schedule (where the
 *       chunked kernel applies; otherwise the token-serial kernel).
 * The two chunked schedules give bit-identical results, so choices 0, 2 and 3 agree bit
 * for bit, and a prompt's results do not depend on the pack around it even where the
 * automatic choice differs; the token-serial kernel agrees with them to rounding. Errors: INVALID_ARGUMENT. */
gdn_status gdn_set_kernel_preference(gdn_handle* handle, int32_t preference);

/* Test hook for the device-side timeout path (hook 1; 0 = off, the default). While it is
 * set, the chunked tensor-core kernels leave out every unit's first q/k tile copy, so each
 * unit's first copy wait runs out after its time bound (about one second of polling) with
 * no fault: the kernel records GDN_ERR_DEVICE_TIMEOUT in the status word that
 * gdn_read_device_status returns, lets every copy and product it did issue land, frees its
 * tensor memory and returns. The outputs of such a call are undefined; the CUDA context
 * stays usable. The token-serial kernel ignores the hook. Errors: INVALID_ARGUMENT. */
gdn_status gdn_set_test_hook(gdn_handle* handle, int32_t hook);

/* The chunked kernel's schedule that the automatic choice takes for a pack of `num_seqs`
 * prompts (cu_seqlens_host: prefix sums, as for gdn_prefill_packed) with `num_v_heads`
 * value heads on a GPU with `num_sms` SMs: *schedule = 2 (pipelined) or 3 (throughput),
 * the gdn_set_kernel_preference codes. The choice is the smaller of two estimates from
 * costs measured on GB300 (microseconds): 5.12 per chunk plus 15.7 per unit for a
 * pipelined unit on its own SM; 8.93 per chunk plus 13.2 per unit for one of two
 * throughput units sharing an SM, 6.38 plus 17.3 for one alone; 8.0 and 16.6 per unit of a
 * prompt with one token or none (which the same launch runs with the decode step's
 * arithmetic) on a pipelined or throughput slot. Over W = the chunks of the U other
 * (prompt, value head) units, Lmax = the chunks of the longest and S = the short units:
 *   pipelined:  max(5.12 Lmax + 15.7, (5.12 W + 15.7 U + 8.0 S) / num_sms,
 *                   ceil(U / num_sms) (5.12 W / U + 15.7))
 *   throughput: max(Lchain, R, (8.93 W + 13.2 U + 16.6 S) / (2 num_sms)), with
 *               Lchain = 8.93 Lmax + 13.2 when U > num_sms, else 6.38 Lmax + 17.3, and
 *               R = F (8.93 W / U + 13.2) + the last round, F = floor(U / (2 num_sms)):
 *               paired (8.93 W / U + 13.2) if its units outnumber the SMs, else alone
 *               (6.38 W / U + 17.3), else nothing
 * (the 15.7 and 17.3 terms and the rounds only when U > 0): a unit never moves between
 * SMs, so a pack runs in whole rounds, and a throughput pack with more units than SMs
 * has SMs running two units at once.
 * Both schedules give bit-identical results; only the time differs. Host-only arithmetic,
 * no CUDA call. Errors: INVALID_ARGUMENT (num_seqs < 0, cu NULL with num_seqs > 0,
 * cu[0] != 0 or decreasing, num_v_heads < 1, num_sms < 1, schedule NULL). */
gdn_status gdn_chunked_schedule(int32_t num_seqs, const int32_t* cu_seqlens_host,
                                int32_t num_v_heads, int32_t num_sms, int32_t* schedule);

/* Device workspace bytes that gdn_prefill_packed needs for this pack (the chunk/tile work
 * list). Validates the same arguments gdn_prefill_packed validates about the pack.
 * Result is a multiple of 256 and at least 256. */
gdn_status gdn_prefill_workspace_size(const gdn_config* cfg, int32_t num_seqs,
                                      const int32_t* cu_seqlens_host,
                                      const int32_t* ckpt_cu_host, size_t* bytes);

/* Packed variable-length prefill of the gated delta rule.
 *
 *  num_seqs         N >= 1 prompts in the pack.
 *  cu_seqlens_host  [N+1] int32, cu[0] = 0, non-decreasing; prompt n is tokens
 *                   [cu[n], cu[n+1]). Zero-length prompts are allowed: their final state
 *                   is their initial state and they emit no output.
 *  q, k             [T][H_k][d] io_dtype.   v: [T][H_v][d] io_dtype.
 *  a, beta          [T][H_v] fp32: log-decay (g = exp(a), a <= 0) and the write strength.
 *                   a = -inf (g = 0) is allowed: the state restarts at that token.
 *  initial_state    [N][H_v][d][d] fp32, or NULL for all-zero initial states.
 *  ckpt_cu_host     [N+1] int32 CSR over ckpt_pos_host (ckpt_cu[0] = 0), or NULL when no
 *                   prompt asks for a checkpoint.
 *  ckpt_pos_host    prompt-relative positions p: the snapshot is the state after the first
 *                   p tokens of that prompt's segment. Per prompt strictly increasing, in
 *                   [1, len], and each a multiple of chunk_size or equal to len
 *                   (otherwise GDN_ERR_UNSUPPORTED).
 *  o                [T][H_v][d] io_dtype output.
 *  ckpt_states      [ckpt_cu[N]][H_v][d][d] fp32; slot j holds checkpoint j of the CSR.
 *                   May be NULL only when there is no checkpoint.
 *  final_states     [N][H_v][d][d] fp32 state after each prompt's last token. May equal
 *                   initial_state (in-place update); no other overlap is allowed.
 *  workspace        device scratch of at least gdn_prefill_workspace_size() bytes,
 *                   256-byte aligned; it must not be reused by other work before this
 *                   call's work on `stream` has finished.
 * The result does not depend on how prompts are packed: each prompt's outputs, checkpoints
 * and final state are bit-identical whether it runs alone or inside any pack ("the same
 * checkpoints whether prompts are prefilled alone or packed", sparkinfer v0.6.28,
 * pack_ckpt_check). Errors: INVALID_ARGUMENT, UNSUPPORTED, WORKSPACE_TOO_SMALL, CUDA. */
gdn_status gdn_prefill_packed(gdn_handle* handle, const gdn_config* cfg, int32_t num_seqs,
                              const int32_t* cu_seqlens_host,
                              const void* q, const void* k, const void* v,
                              const float* a, const float* beta,
                              const float* initial_state,
                              const int32_t* ckpt_cu_host, const int32_t* ckpt_pos_host,
                              void* o, float* ckpt_states, float* final_states,
                              void* workspace, size_t workspace_bytes, void* stream);

/* Host image of the work list that gdn_prefill_packed would upload for this pack and
 * handle (handle may be NULL: automatic kernel choice), for inspection and tests. Layout,
 * each array on a 256-byte boundary: int32 status, int32 num_units, then num_units units
 * {int32 seq, head, row0, nrows} ordered longest prompt first, then per-prompt records
 * {int32 tok_start, len, ckpt_begin, ckpt_end, flags, state_slot}, then the checkpoint
 * positions, then one int32 per prompt (zero: the checkpoint counters that
 * gdn_prefill_packed_snapshot's kernels count up).
 * *bytes_needed receives the size; with out == NULL nothing else is written. Errors as
 * gdn_prefill_packed's pack checks, or WORKSPACE_TOO_SMALL when out_bytes is short. */
gdn_status gdn_prefill_worklist_host(gdn_handle* handle, const gdn_config* cfg,
                                     int32_t num_seqs, const int32_t* cu_seqlens_host,
                                     const int32_t* ckpt_cu_host, const int32_t* ckpt_pos_host,
                                     void* out, size_t out_bytes, size_t* bytes_needed);

/* Read the device status word that the last prefill using `workspace` left behind (0 when
 * every bounded device-side wait completed, GDN_ERR_DEVICE_TIMEOUT when one gave up).
 * Synchronises `stream`. Errors: INVALID_ARGUMENT, CUDA. */
gdn_status gdn_read_device_status(const void* workspace, int32_t* status_out, void* stream);

/* Copy `bytes` of device checkpoint states into the handle's pinned pool at byte offset
 * `pool_offset`, on the handle's side stream, after all work already queued on `stream`
 * (so the scan and the copy of the next prompts overlap; sparkinfer v0.6.28, bullet on
 * separate streams for the scan and the checkpoint copy). Returns at once; completion is
 * observed with gdn_checkpoint_copy_query / _wait. Errors: INVALID_ARGUMENT,
 * POOL_EXHAUSTED (range outside the pool), CUDA. */
gdn_status gdn_checkpoint_copy(gdn_handle* handle, const float* ckpt_states_dev, size_t bytes,
                               size_t pool_offset, void* stream);

/* gdn_prefill_packed whose checkpoints are copied into the handle's pinned pool while the
 * scan still runs ("the scan and the checkpoint copy run on separate streams, not one after
 * another", sparkinfer v0.6.28 release notes, bullet 2; the pool itself: bullet on pinned
 * host buffers). Checkpoint slot j lands at byte pool_offset + j * H_v * d * d * 4 of the
 * pool, the same layout as ckpt_states. Every block of the launch counts its prompt's
 * stored checkpoints in a per-prompt counter in the workspace; on the handle's side
 * stream, each copy of a run of prompts (consecutive prompt indices in the work list's
 * longest-first order, up to 8 MiB) first waits on the device until its prompts' counters
 * are complete (cuStreamWaitValue32), so the snapshots of prompts that finish early leave
 * while later prompts are still in the scan. Where the driver offers no stream wait on
 * memory, one copy follows the whole pass. Outputs are bit-identical to gdn_prefill_packed's.
 * Completion: gdn_checkpoint_copy_query / _wait on the host, gdn_checkpoint_copy_event or
 * gdn_checkpoint_copy_join on the device. Arguments and errors as gdn_prefill_packed, plus
 * POOL_EXHAUSTED when the checkpoints do not fit in the pool at pool_offset. The workspace
 * must not be reused before the copies have completed. */
gdn_status gdn_prefill_packed_snapshot(gdn_handle* handle, const gdn_config* cfg,
                                       int32_t num_seqs, const int32_t* cu_seqlens_host,
                                       const void* q, const void* k, const void* v,
                                       const float* a, const float* beta,
                                       const float* initial_state,
                                       const int32_t* ckpt_cu_host, const int32_t* ckpt_pos_host,
                                       void* o, float* ckpt_states, float* final_states,
                                       size_t pool_offset, void* workspace,
                                       size_t workspace_bytes, void* stream);

/* GDN_OK when every checkpoint copy issued so far has completed, otherwise
 * GDN_ERR_DEVICE_TIMEOUT (not finished yet; nothing is wrong). */
gdn_status gdn_checkpoint_copy_query(gdn_handle* handle);

/* Block the calling host thread until every checkpoint copy issued so far has completed. */
gdn_status gdn_checkpoint_copy_wait(gdn_handle* handle);

/* The device-side completion of the checkpoint copies (the scan and the copy on separate
 * streams, sparkinfer v0.6.28 release notes, bullet 2): *event_out receives the handle's
 * cudaEvent_t (as void*), recorded on the side stream after the last copy issued so far
 * by gdn_checkpoint_copy or gdn_prefill_packed_snapshot, so that a consumer stream can
 * order itself after the snapshots without blocking a host thread
 * (cudaStreamWaitEvent). The handle owns the event; every later copy call records it
 * again, so take it after the copies it should cover have been issued. Before any copy it
 * has never been recorded, and a wait on it completes at once. Errors: INVALID_ARGUMENT. */
gdn_status gdn_checkpoint_copy_event(gdn_handle* handle, void** event_out);

/* Make `stream` wait on the device for every checkpoint copy issued so far (the same
 * ordering as a cudaStreamWaitEvent on gdn_checkpoint_copy_event's event); returns at
 * once. Errors: INVALID_ARGUMENT, CUDA. */
gdn_status gdn_checkpoint_copy_join(gdn_handle* handle, void* stream);

/* Prefill on the handle's own stream, so that a prefill pass overlaps decode steps that
 * keep running on the caller's streams ("run at most one in-flight prefill on an owned
 * CUDA stream", pegainfer PR #786, Changes). Arguments as gdn_prefill_packed; the owned
 * stream first waits for the work already queued on `after_stream` (the inputs'
 * producer), then runs the prefill and records a completion event. At most one prefill
 * is in flight per handle: while the previous one runs, the call returns GDN_ERR_BUSY
 * and enqueues nothing. Completion: gdn_prefill_async_query (poll), _wait (block the
 * host) or _join (make another stream wait on the device). gdn_handle_destroy drains the
 * owned stream first. */
gdn_status gdn_prefill_packed_async(gdn_handle* handle, const gdn_config* cfg,
                                    int32_t num_seqs, const int32_t* cu_seqlens_host,
                                    const void* q, const void* k, const void* v,
                                    const float* a, const float* beta,
                                    const float* initial_state,
                                    const int32_t* ckpt_cu_host, const int32_t* ckpt_pos_host,
                                    void* o, float* ckpt_states, float* final_states,
                                    void* workspace, size_t workspace_bytes,
                                    void* after_stream);

/* GDN_OK when no prefill is in flight on the handle's stream (the last one completed),
 * GDN_ERR_DEVICE_TIMEOUT while it is still running ("poll completion events while
 * decode is active", pegainfer PR #786). */
gdn_status gdn_prefill_async_query(gdn_handle* handle);

/* Block the host until the in-flight prefill (if any) has completed ("wait explicitly
 * when the last decoder retires", pegainfer PR #786). */
gdn_status gdn_prefill_async_wait(gdn_handle* handle);

/* Make `stream` wait on the device for the in-flight prefill (if any); returns at once. */
gdn_status gdn_prefill_async_join(gdn_handle* handle, void* stream);

/* One-token decode update for `batch` decoding sequences, each with its own fp32 state in
 * a caller-owned pool, updated in place (vllm.cpp "vLLM, online serving", packed GDN
 * decode lever). For sequence b:
 *     S = state_pool[slot_idx[b]]   ([H_v][d][d] fp32 per slot)
 *     one step of the recurrence with q[b], k[b] ([batch][H_k][d]), v[b] ([batch][H_v][d]),
 *     a[b], beta[b] ([batch][H_v] fp32); o[b] ([batch][H_v][d] io_dtype) = scale * S_new q
 *  slot_idx_dev     [batch] int32 device array of distinct slot indices in [0, num_slots).
 * Distinct slots are the caller's duty (two batch rows naming one slot race).
 * The call checks its arguments on the host and enqueues one kernel on `stream`, with no
 * copy and no allocation, so a serving loop can capture it in a CUDA graph and replay it
 * (the graph then keeps the buffer addresses of the capture; a test replays captured
 * steps and matches direct calls bit for bit).
 * Errors: INVALID_ARGUMENT, UNSUPPORTED, CUDA. */
gdn_status gdn_decode_step(gdn_handle* handle, const gdn_config* cfg, int32_t batch,
                           const void* q, const void* k, const void* v,
                           const float* a, const float* beta,
                           float* state_pool, int32_t num_slots, const int32_t* slot_idx_dev,
                           void* o, void* stream);

/* Bytes of the fixed device scratch behind gdn_prefill_packed_noalloc (per GPU). */
#define GDN_NOALLOC_SCRATCH_BYTES (1u << 20)

/* gdn_prefill_packed for callers that cannot allocate memory when they call in: there is
 * no workspace and no handle argument, and nothing is allocated. The pages describe no
 * such call; it exists for serving engines whose device memory is all handed to their own
 * pool at start-up, and for plugins whose host framework forbids allocation on the request
 * path. Arguments, layouts, results and errors are those of gdn_prefill_packed, except
 * that a device-side timeout is read with gdn_noalloc_read_status (gdn_read_device_status
 * needs a workspace).
 * The work list lives in one file-scope device array of GDN_NOALLOC_SCRATCH_BYTES per GPU
 * (held from library load to process exit); a pack whose work list does not fit returns
 * GDN_ERR_UNSUPPORTED before anything is enqueued. Every call rewrites that array and
 * clears its status word, so calls whose device work may overlap in time (two streams)
 * race and must be serialised by the caller. The first call on each device looks up the
 * array's device address (cudaGetSymbolAddress) with that device current; make that
 * first call before any stream capture. That address belongs to the device's primary
 * context: after a cudaDeviceReset in the same process, do not use this entry point. The
 * host copy of the work list is taken from one fixed host buffer under one process-wide
 * lock with a pageable cudaMemcpyAsync, so a call may block the host until work queued
 * earlier on `stream` has drained, and calls on different GPUs run one after another. */
gdn_status gdn_prefill_packed_noalloc(const gdn_config* cfg, int32_t num_seqs,
                                      const int32_t* cu_seqlens_host,
                                      const void* q, const void* k, const void* v,
                                      const float* a, const float* beta,
                                      const float* initial_state,
                                      const int32_t* ckpt_cu_host, const int32_t* ckpt_pos_host,
                                      void* o, float* ckpt_states, float* final_states,
                                      void* stream);

/* Mixed step in one launch, with the states gathered from a pool (sparkinfer v0.6.4 release
 * notes, "What changed": prompt slices under a 1,024-token budget run in the same pass as
 * the decoding requests; vllm.cpp "vLLM, online serving", lever 2b, packed GDN decode).
 * gdn_prefill_packed in which every prompt's state lives in a caller-owned pool and is
 * updated in place: prompt n reads its initial state from state_pool[slot_idx_host[n]]
 * (or starts from a zero state when start_zero_host is non-NULL and start_zero_host[n] !=
 * 0) and writes its final state back to the same slot. Decoding sequences ride the pack as
 * one-token prompts; every (prompt, value head) unit, prompts of one token or none
 * included, runs in one kernel launch (gdn_prefill_launch_count reports it), so a mixed
 * step of prompt slices and decode tokens needs no caller-side state copies and no second
 * launch.
 *  state_pool       [num_slots][H_v][d][d] fp32 device, 16-byte aligned; slots not named by
 *                   slot_idx_host are neither read nor written.
 *  slot_idx_host    [N] int32 host array of distinct slots in [0, num_slots).
 *  start_zero_host  [N] int32 host array or NULL (NULL: every prompt reads its slot).
 * Everything else as gdn_prefill_packed (the workspace size is gdn_prefill_workspace_size's).
 * The pool may not overlap q, k, v, a, beta, o, ckpt_states or the workspace. Errors:
 * INVALID_ARGUMENT (also for a slot out of range or named twice), UNSUPPORTED,
 * WORKSPACE_TOO_SMALL, CUDA. */
gdn_status gdn_prefill_packed_pool(gdn_handle* handle, const gdn_config* cfg, int32_t num_seqs,
                                   const int32_t* cu_seqlens_host,
                                   const void* q, const void* k, const void* v,
                                   const float* a, const float* beta,
                                   float* state_pool, int32_t num_slots,
                                   const int32_t* slot_idx_host, const int32_t* start_zero_host,
                                   const int32_t* ckpt_cu_host, const int32_t* ckpt_pos_host,
                                   void* o, float* ckpt_states,
                                   void* workspace, size_t workspace_bytes, void* stream);

/* Number of kernels that the handle's last prefill call (gdn_prefill_packed and its _pool,
 * _snapshot, _async, _host and _split forms) enqueued: 1 for any pack of
 * gdn_prefill_packed, gdn_prefill_packed_pool or gdn_prefill_packed_snapshot with at least
 * one prompt. Host-side bookkeeping (no CUDA call). Errors: INVALID_ARGUMENT. */
gdn_status gdn_prefill_launch_count(gdn_handle* handle, int32_t* count);

/* The status word that the last gdn_prefill_packed_noalloc call on the current device
 * left (0, or GDN_ERR_DEVICE_TIMEOUT when a bounded device-side wait gave up) into
 * *status_out: a copy from the fixed device array into the caller's int32 on `stream`,
 * which it synchronises. No allocation. The pages have no counterpart. Errors:
 * INVALID_ARGUMENT, UNSUPPORTED (device index beyond 63), CUDA. */
gdn_status gdn_noalloc_read_status(int32_t* status_out, void* stream);

/* Process-wide test hook of gdn_prefill_packed_noalloc for the device-side timeout path,
 * with the meaning of gdn_set_test_hook's hook 1 (0 = off, the default). The pages have no
 * counterpart. Errors: INVALID_ARGUMENT. */
gdn_status gdn_noalloc_set_test_hook(int32_t hook);

/* ---- prefill from host memory ---------------------------------------------------------- */

/* The arrays of one pack, in the layouts of gdn_prefill_packed: inputs q, k, v, a, beta and
 * initial_state (NULL = zeros), outputs o, ckpt_states (NULL when the pack has no
 * checkpoints) and final_states. */
typedef struct {
  void* q;
  void* k;
  void* v;
  float* a;
  float* beta;
  float* initial_state;
  void* o;
  float* ckpt_states;
  float* final_states;
} gdn_prefill_buffers;

/* gdn_prefill_packed for a pack whose inputs and outputs live in host memory. The prompts
 * are processed in groups of up to `group_prompts`: the groups grow 1, 2, 4, ... prompts up
 * to group_prompts at the start and shrink the same way at the end, which keeps short the
 * copy-in that precedes the first prefill and the copy-out that follows the last one. A
 * group's rows of q, k, v, a, beta and its
 * initial states are copied into `device` on the handle's copy-in stream; its prefill runs
 * on `stream` (exactly as gdn_prefill_packed over that group); its o rows, checkpoints and
 * final states are copied back into `host` on the handle's copy-out stream. The copies of
 * neighbouring groups therefore overlap each other and the prefill: about the larger of
 * the two copy volumes over the link rather than their sum. `stream` waits for the last
 * copy out before anything queued after the call. Host buffers should be pinned
 * (cudaHostAlloc) for full copy speed; `device` buffers are the pack-sized device arrays
 * gdn_prefill_packed would take (their inputs are overwritten with the host inputs).
 * Validation is that of gdn_prefill_packed on the whole pack and on `device`. Errors: also
 * INVALID_ARGUMENT for a missing host array or group_prompts < 1, UNSUPPORTED for more than
 * 64 groups. Results equal gdn_prefill_packed's on the whole pack bit for bit (a prompt's
 * results do not depend on its pack, and both chunked schedules agree bit for bit). The
 * workspace holds every group's work list, uploaded in one copy ahead of the bulk copies
 * (gdn_prefill_host_workspace_size). */
/* Device workspace bytes that gdn_prefill_packed_host needs for this pack and group size
 * (the work lists of all groups). A multiple of 256. */
gdn_status gdn_prefill_host_workspace_size(const gdn_config* cfg, int32_t num_seqs,
                                           const int32_t* cu_seqlens_host,
                                           const int32_t* ckpt_cu_host, int32_t group_prompts,
                                           size_t* bytes);

gdn_status gdn_prefill_packed_host(gdn_handle* handle, const gdn_config* cfg,
                                   int32_t num_seqs, const int32_t* cu_seqlens_host,
                                   const int32_t* ckpt_cu_host, const int32_t* ckpt_pos_host,
                                   const gdn_prefill_buffers* host,
                                   const gdn_prefill_buffers* device, int32_t group_prompts,
                                   void* workspace, size_t workspace_bytes, void* stream);

/* ---- sequence splitting ------------------------------------------------------------ */

/* Device workspace bytes that gdn_prefill_packed_split needs for this pack and segment
 * length (work lists of its two passes plus fp32 scratch states: two per segment map and
 * two per split segment). Validates what gdn_prefill_packed_split validates about the
 * pack. Result is a multiple of 256. */
gdn_status gdn_prefill_split_workspace_size(const gdn_config* cfg, int32_t num_seqs,
                                            const int32_t* cu_seqlens_host,
                                            const int32_t* ckpt_cu_host,
                                            const int32_t* ckpt_pos_host, int32_t segment_len,
                                            size_t* bytes);

/* gdn_prefill_packed with prompts longer than `segment_len` tokens cut into segments of
 * `segment_len` (a multiple of 64, >= 64) that run in parallel: more (segment, value head)
 * units for packs with few prompts, such as one very long prompt. The recurrence is affine
 * in a segment's initial state, S_end = S_start M + B; pass 1 computes, for every middle
 * segment, B (from a zero state) and M (from the identity with v taken as zero) next to
 * segment 0 of every prompt; a scan composes the maps in fp32 into each segment's initial
 * state; pass 2 runs segments 1 .. P-1 from those states with their checkpoints. The work
 * is about (2P - 1) / P times that of one pass, in about 2 / P of its sequential chunks.
 * Arguments, layouts and errors are those of gdn_prefill_packed plus `segment_len`
 * (INVALID_ARGUMENT when it is not a positive multiple of 64). Results equal
 * gdn_prefill_packed's to rounding: the composed state carries the maps' fp32 rounding
 * and the fp16 tensor-core operands of each run (the same tolerance applies). Prompts
 * of at most `segment_len` tokens run exactly as in gdn_prefill_packed. `o` is written
 * twice for middle segments (the first write is scratch). */
gdn_status gdn_prefill_packed_split(gdn_handle* handle, const gdn_config* cfg,
                                    int32_t num_seqs, const int32_t* cu_seqlens_host,
                                    const void* q, const void* k, const void* v,
                                    const float* a, const float* beta,
                                    const float* initial_state, const int32_t* ckpt_cu_host,
                                    const int32_t* ckpt_pos_host, void* o, float* ckpt_states,
                                    float* final_states, int32_t segment_len, void* workspace,
                                    size_t workspace_bytes, void* stream);

/* The segment length for gdn_prefill_packed_split that the chunked kernels' cost model
 * (the per-chunk costs of gdn_chunked_schedule) expects to run this pack fastest, or 0 when
 * splitting is not expected to pay (then call gdn_prefill_packed). It compares the whole
 * pack in one launch with P = 2 .. 16 segments of the longest prompt (each a multiple of
 * 64): pass 1 with segment 0 of every prompt plus two map runs per middle segment, pass 2
 * with the later segments, and 12 us for the extra launches. Splitting shortens the longest
 * chain of chunks, so it pays for packs with few (prompt, value head) units per SM and one
 * long prompt, such as one 32K prompt or a ragged pack with one long prompt; the choice
 * depends on the whole pack, so results split this way carry the split path's rounding
 * (gdn_prefill_packed_split) rather than being bit-identical to gdn_prefill_packed's.
 * Host-only, no CUDA call. Errors: INVALID_ARGUMENT (as gdn_chunked_schedule). */
gdn_status gdn_split_segment_auto(int32_t num_seqs, const int32_t* cu_seqlens_host,
                                  int32_t num_v_heads, int32_t num_sms, int32_t* segment_len);

/* ---- full-attention layers: paged 8-bit key/value cache ------------------------------ */

/* The hybrid models whose linear layers the calls above serve interleave them with full
 * attention layers. These calls are the serving side of such a layer: one plan per step
 * (pages and slots of the step's tokens, built on the GPU so that a step needs no host
 * lengths and can be captured in a CUDA graph), then per layer a rotary embedding, an append
 * that quantises keys and values into a paged cache, and the attention that reads it.
 *
 * Conventions: a request's tokens are numbered from 0; page p of a request holds its tokens
 * [p * page_size, (p + 1) * page_size); block_table [num_seqs][max_blocks] int32 (device)
 * gives each request's pages in order. A token's slot is page * page_size + its place in the
 * page. Lengths, tables and slots live on the device and are checked there: a value out of
 * range is never used as an address. Where `status` is a non-NULL device int32, the kernels
 * raise it (atomic maximum) to GDN_ERR_INVALID_ARGUMENT when they met such a value; they
 * never clear it, so a caller zeroes it once and reads it when it likes. A bounded device
 * wait that gave up raises it to GDN_ERR_DEVICE_TIMEOUT. */

/* A paged cache of e4m3 values with one fp32 scale for each page and head. A cached value is
 * its e4m3 code times its page's and head's scale; v holds no NaN codes (gdn_kv_append puts a
 * token's NaN into its key alone). All arrays are device memory, k and v
 * 16-byte aligned. Supported: page_size 16, 32, 64 or 128, head_dim 64, 128 or 256,
 * num_pages * num_kv_heads * page_size <= INT32_MAX. */
typedef struct gdn_kv_cache {
  int32_t num_pages;
  int32_t page_size;     /* tokens of a page */
  int32_t num_kv_heads;
  int32_t head_dim;
  void* k;               /* [num_pages][num_kv_heads][page_size][head_dim] e4m3 */
  void* v;               /* the same layout */
  float* k_scale;        /* [num_pages][num_kv_heads], each finite and >= 0 */
  float* v_scale;
} gdn_kv_cache;

/* Pages and slots of one step, built on the GPU (one kernel). Request b has ctx_len[b]
 * tokens in the cache, in the first ceil(ctx_len[b] / page_size) entries of its table row,
 * and appends new_len[b] tokens, whose rows follow one another in request order. Requests are
 * served in order: each takes the pages that its new tokens need beyond the ones it has from
 * the top of the free stack free_pages[0 .. *free_count) (the top is the last entry), and
 * they are written behind its present ones in its table row.
 *  num_tokens       rows of the step's arrays (at least the sum of new_len).
 *  free_count       [1] pages on the stack. free_count_out [1] receives what is left; it may
 *                   be free_count itself.
 *  cu_new           [num_seqs + 1] out: first row of every request, then the number of rows.
 *  kv_len           [num_seqs] out: ctx_len + new_len, the lengths the attention takes.
 *  positions        [num_tokens] out (or NULL): the rows' positions, ctx_len[b] + i; 0 past
 *                   the last row.
 *  slots            [num_tokens] int64 out: the rows' slots; -1 past the last row.
 * A request that cannot be served takes no page: its kv_len is 0 and its slots are -1 (the
 * append then stores nothing for it, and the attention gives it zeros), and status is raised
 * to GDN_ERR_POOL_EXHAUSTED when the stack ran out (no later request that needs a page is
 * served then), or to GDN_ERR_INVALID_ARGUMENT for lengths below 0, more pages than
 * max_blocks, rows past num_tokens, or a page out of range: the half-filled one that its first
 * new tokens go to, or one on the stack (the stack counts as ending in front of it, so no later
 * request that needs a page is served either). A caller keeps such a request's ctx_len as it
 * was: its table row is untouched. At most 4,096 requests.
 * Errors: INVALID_ARGUMENT, UNSUPPORTED, CUDA. */
gdn_status gdn_kv_plan(gdn_handle* handle, int32_t page_size, int32_t num_seqs,
                       int32_t num_tokens, const int32_t* ctx_len, const int32_t* new_len,
                       int32_t* block_table, int32_t max_blocks, int32_t num_pages,
                       const int32_t* free_pages, const int32_t* free_count,
                       int32_t* free_count_out, int32_t* cu_new, int32_t* kv_len,
                       int32_t* positions, int64_t* slots, int32_t* status, void* stream);

/* Give back the pages of requests that ended (one kernel): for every b with release[b] != 0,
 * in order, the ceil(kv_len[b] / page_size) pages of its table row are pushed on the free
 * stack and its table entries become -1. A row with a page out of range, or whose pages would
 * overfill the stack (num_pages entries), is left as it is and raises the status.
 * Errors: INVALID_ARGUMENT, UNSUPPORTED (more than 4,096 requests), CUDA. */
gdn_status gdn_kv_release(gdn_handle* handle, int32_t page_size, int32_t num_seqs,
                          const int32_t* kv_len, const int32_t* release, int32_t* block_table,
                          int32_t max_blocks, int32_t num_pages, int32_t* free_pages,
                          int32_t* free_count, int32_t* status, void* stream);

#define GDN_ROPE_MAX_PAIRS 128
#define GDN_ROPE_MAX_AXES 4

/* How the rotated pairs are shared out among the axes: whole sections one after another, or
 * in turns (pair i belongs to axis i mod num_axes while that axis has pairs left, the rest
 * and the turns of exhausted axes to axis 0). */
typedef enum gdn_rope_axes { GDN_ROPE_SECTIONS = 0, GDN_ROPE_INTERLEAVED = 1 } gdn_rope_axes;
/* Which elements form pair i of a rotary part of R elements: (i, i + R/2) or (2i, 2i + 1). */
typedef enum gdn_rope_pairs { GDN_ROPE_HALVES = 0, GDN_ROPE_ADJACENT = 1 } gdn_rope_pairs;

/* A rotary embedding, filled once by gdn_rope_init. A frequency is kept as the 64-bit
 * fraction of a turn per position, so that position * frequency modulo a turn is one integer
 * product, exact to 2^-33 of a turn for every int32 position. */
typedef struct gdn_rope {
  int32_t head_dim;
  int32_t rotary_dim;   /* R: the first R elements of a head are rotated, the rest pass */
  int32_t num_axes;
  int32_t pair_layout;  /* gdn_rope_pairs */
  uint64_t turns[GDN_ROPE_MAX_PAIRS];  /* pair i: frequency / (2 pi), times 2^64 */
  uint8_t axis[GDN_ROPE_MAX_PAIRS];    /* pair i: the axis whose position it follows */
} gdn_rope;

/* Fill a gdn_rope. sections[num_axes]: pairs of each axis (time, height, width, ...), their
 * sum R/2. inv_freq: R/2 angular frequencies (radians per position, each in [0, 2 pi)), or
 * NULL for theta^(-2i/R). Supported: head_dim 64, 128 or 256, rotary_dim a multiple of 16
 * up to head_dim, 1 to 4 axes. Host arithmetic, no CUDA call. Errors: INVALID_ARGUMENT,
 * UNSUPPORTED. */
gdn_status gdn_rope_init(gdn_rope* rope, int32_t head_dim, int32_t rotary_dim,
                         int32_t num_axes, const int32_t* sections, int32_t axis_layout,
                         int32_t pair_layout, double theta, const double* inv_freq);

/* Rotate the heads of q and k (one kernel): pair (x, y) with angle w = position[axis] *
 * frequency becomes (x cos w - y sin w, y cos w + x sin w), in fp32, rounded once.
 *  positions  [num_axes][pos_stride] int32 (device): row `a` holds the tokens' positions on
 *             axis a; any int32 value.
 *  q, q_out   token t's heads at q + t * q_stride (elements), [num_q_heads][head_dim]
 *             contiguous; q_out the same with its own stride. q_out may be q with the same
 *             stride (in place); no other overlap. num_q_heads 0: no q. The same for k.
 * Pointers 16-byte aligned, strides multiples of 16 bytes and at least heads * head_dim (so
 * q and k may be column ranges of one projection's output). Errors: INVALID_ARGUMENT, CUDA. */
gdn_status gdn_rope_apply(gdn_handle* handle, const gdn_rope* rope, int32_t io_dtype,
                          int32_t num_tokens, const int32_t* positions, int64_t pos_stride,
                          const void* q, int64_t q_stride, int32_t num_q_heads, void* q_out,
                          int64_t q_out_stride, const void* k, int64_t k_stride,
                          int32_t num_k_heads, void* k_out, int64_t k_out_stride, void* stream);

/* Quantise the step's keys and values into the cache (one kernel). Row t goes to slots[t]
 * ([num_tokens] int64, device; a negative slot is skipped). Rows of one page must follow one
 * another with rising slots, as gdn_kv_plan numbers them, and what the page holds in front of
 * the first of them must be the request's earlier tokens; the call's rows name each page in
 * one such run only.
 * A page's and head's scale is the least power of two s with |x| <= 448 s for every finite
 * value it has held since its first token (2^-100 at least): it never shrinks while the page
 * fills, and when it grows the codes in front are rounded to it (exact but for the smallest,
 * since only their exponent moves). A run that begins at the page's first token starts the
 * scale anew. Values are rounded to the nearest e4m3, ties to even; infinities are held as
 * the largest finite value; a NaN in k stays NaN, and a token with a NaN in v gets a NaN key
 * and zeros for its NaN values: such a token makes NaN every output that attends to it and
 * no other.
 *  k, v       token t's heads at k + t * k_stride (elements), [num_kv_heads][head_dim].
 *  rope       NULL: k is stored as given. Otherwise k is rotated on the way (in fp32, one
 *             rounding), and when num_q_heads > 0 so is q into q_out, as gdn_rope_apply.
 * Alignment and strides as gdn_rope_apply. Errors: INVALID_ARGUMENT, UNSUPPORTED, CUDA. */
gdn_status gdn_kv_append(gdn_handle* handle, const gdn_kv_cache* cache, int32_t io_dtype,
                         int32_t num_tokens, const int64_t* slots, const void* k,
                         int64_t k_stride, const void* v, int64_t v_stride,
                         const gdn_rope* rope, const int32_t* positions, int64_t pos_stride,
                         const void* q, int64_t q_stride, int32_t num_q_heads, void* q_out,
                         int64_t q_out_stride, int32_t* status, void* stream);

/* Attention over the paged cache. */
typedef struct gdn_attn_config {
  int32_t num_q_heads;  /* a multiple of the cache's num_kv_heads; query head h reads
                           key/value head h / (num_q_heads / num_kv_heads) */
  int32_t causal;       /* nonzero: query i of a request with q_len queries and kv_len cached
                           tokens sees tokens 0 .. kv_len - q_len + i; zero: all of them */
  int32_t io_dtype;     /* gdn_dtype of q and o */
  float scale;          /* of the scores, usually 1/sqrt(head_dim) */
} gdn_attn_config;

/* Device workspace of gdn_attn_paged for calls of at most these sizes (multiple of 256). */
gdn_status gdn_attn_workspace_size(const gdn_attn_config* cfg, const gdn_kv_cache* cache,
                                   int32_t num_seqs, int32_t num_tokens, int32_t max_q_len,
                                   int32_t max_kv_len, size_t* bytes);

/* o = softmax(scale q K^T) V for a pack of requests of any mix of lengths: decoding requests
 * (one query), drafts (a few) and prompts, behind any cached prefix. K and V are the cached
 * tokens, the call's own among them (append first).
 *  num_tokens   rows of q, o and lse.
 *  max_q_len, max_kv_len  host bounds of the requests' lengths: they choose the kernels and
 *               the split of the work; a longer request is cut to them (status raised).
 *  cu_q         [num_seqs + 1] device: request b's queries are rows [cu_q[b], cu_q[b+1]).
 *  kv_len       [num_seqs] device: its cached tokens (0 is allowed).
 *  q, o         token t's heads at q + t * q_stride (elements), [num_q_heads][head_dim].
 *  lse          [num_tokens][num_q_heads] fp32 out, or NULL: log of the sum of exponentials.
 * A query that sees no token gives o = 0 and lse = -inf. Pages out of range count as absent
 * (status raised). Rows outside every request are not written; requests that overlap (cu_q out
 * of order, status raised) write their common rows in any order, and nothing is written where
 * together they ask for 2^31 work items.
 * Scores, softmax sums and outputs are accumulated in fp32. The cache's codes enter the products
 * exactly, and so do bf16 queries, but for values below 2^-10 of their row's largest where a
 * request has many queries: those are off by at most 2^-17 of the largest. A token's weight, its probability times its
 * value scale, is rounded to fp16's 11 bits, or to 2^-31 of the largest weight of its row where
 * that is more: tokens that a row does not see, or gives no weight, change nothing of it. With
 * fp32 io queries and weights are two fp16 terms, 22 bits (weights to 2^-31 of the row's
 * largest). Value scales below 2^-100 count as 0 and those above 2^120 as 2^120 (gdn_kv_append
 * keeps them in that range). Results do not depend on atomics: the same call gives the same bits.
 * UNSUPPORTED: more than 4,096 requests, 2^31 or more query rows of a key/value head, or more than
 * 2^31 work items, for which every 8 query rows count max_kv_len / 64 + 1 times num_kv_heads: with
 * fp32 io all rows (a prompt of 131,072 tokens over as many, 16 query and 2 key/value heads, is
 * within), with bf16 at most 256 (or twice the heads of a group) of each request.
 * Errors: INVALID_ARGUMENT, UNSUPPORTED, WORKSPACE_TOO_SMALL, CUDA. */
gdn_status gdn_attn_paged(gdn_handle* handle, const gdn_attn_config* cfg,
                          const gdn_kv_cache* cache, int32_t num_seqs, int32_t num_tokens,
                          int32_t max_q_len, int32_t max_kv_len, const int32_t* cu_q,
                          const int32_t* kv_len, const int32_t* block_table,
                          int32_t max_blocks, const void* q, int64_t q_stride, void* o,
                          int64_t o_stride, float* lse, void* workspace,
                          size_t workspace_bytes, int32_t* status, void* stream);

/* ---- around the recurrent layers: convolution, selective scan, norm, sampling ---------- */

/* The rest of a hybrid model's serving step. In front of a recurrent layer (the gated delta rule
 * above, or the selective scan here) stands a short causal convolution over its channels; its
 * output passes a root-mean-square norm, and so does the residual stream in front of every
 * projection, which may take it in 8 bits; the last projection's logits are sampled. Serving
 * forms only, like every call of this library.
 *
 * Requests of the two packed calls are given on the device, as gdn_kv_plan's, so that a step can
 * be captured in a CUDA graph: request n is rows [cu[n], cu[n+1]) and its state lives in slot
 * slot_idx[n] of the caller's pool, where it is updated in place. Any mix of prompts and single
 * tokens is served. A request whose rows or slot are out of range, or that is longer than max_len,
 * is refused whole (nothing of it is read or written); a slot below 0 skips its request. A request
 * that gdn_kv_plan refused (kv_len 0) may have rows in cu all the same: give it such a slot for its
 * state to stay as it was. Rows outside every request served are not written. Where `status` is a non-NULL device int32 the
 * kernels raise it (atomic maximum) to GDN_ERR_INVALID_ARGUMENT when they refused something; they
 * never clear it. Distinct slots and disjoint rows are the caller's duty: requests that share a
 * slot or rows (cu out of order, status raised) race for them, and some of them may be left out. */
typedef struct gdn_requests {
  int32_t num_seqs;          /* 1 .. 4,096 requests                                          */
  int32_t num_tokens;        /* rows of the call's arrays, cu[num_seqs] or more, below
                                2^31 - 4,096                                                 */
  int32_t max_len;           /* host bound of the requests' lengths                          */
  int32_t num_slots;         /* slots of the state pool                                      */
  const int32_t* cu;         /* [num_seqs + 1] first rows; a request of no rows is allowed   */
  const int32_t* slot_idx;   /* [num_seqs], or NULL: request n uses slot n                   */
  const int32_t* start_zero; /* [num_seqs] nonzero: start from zeros, not from the slot; NULL:
                                every request starts from its slot                           */
  const int32_t* ckpt_cu;    /* [num_seqs + 1] CSR over ckpt_pos, or NULL: no checkpoints    */
  const int32_t* ckpt_pos;   /* positions p in [1, length], rising within a request: checkpoint
                                j receives the state after the request's first p rows        */
  int32_t num_ckpt;          /* checkpoints the arrays hold (others are refused)             */
} gdn_requests;

typedef enum gdn_activation { GDN_ACT_NONE = 0, GDN_ACT_SILU = 1 } gdn_activation;

/* Causal convolution of each channel by itself:
 *     y[t][c] = act(bias[c] + sum_j weight[c][j] * x[t - width + 1 + j][c])
 * summed in fp32 and rounded once. Rows in front of a request's first come from its state: the
 * last width - 1 inputs of the request so far, oldest first, [width - 1][channels] io_dtype. */
typedef struct gdn_conv_config {
  int32_t channels;     /* C, 1 .. 262,144 */
  int32_t width;        /* taps, 2 .. 4 */
  int32_t activation;   /* gdn_activation; silu(v) = v / (1 + exp(-v)) */
  int32_t io_dtype;     /* gdn_dtype of x, y and the states */
  const float* weight;  /* [C][width] device; the last tap multiplies the current row */
  const float* bias;    /* [C] device, or NULL */
} gdn_conv_config;

/* The convolution of a pack of requests (one kernel).
 *  x, y        row t's channels at x + t * x_stride (elements); no overlap of x and y.
 *  state_pool  [num_slots][width - 1][C] io_dtype, updated in place.
 *  ckpt_states [num_ckpt][width - 1][C] io_dtype, or NULL without checkpoints.
 * Pointers 16-byte aligned, strides multiples of 16 bytes and at least C (so x may be a column
 * range of a projection's output). Results do not depend on the pack around a request.
 * Errors: INVALID_ARGUMENT, UNSUPPORTED (width, channels, more requests or rows), CUDA. */
gdn_status gdn_conv_packed(gdn_handle* handle, const gdn_conv_config* cfg,
                           const gdn_requests* req, const void* x, int64_t x_stride, void* y,
                           int64_t y_stride, void* state_pool, void* ckpt_states,
                           int32_t* status, void* stream);

/* One token of `batch` decoding requests (one kernel): row b with the state in slot slot_idx[b]
 * (device; below 0: the row is skipped; slots distinct). y may be x with the same stride.
 * Otherwise as gdn_conv_packed. */
gdn_status gdn_conv_step(gdn_handle* handle, const gdn_conv_config* cfg, int32_t batch,
                         const void* x, int64_t x_stride, void* y, int64_t y_stride,
                         void* state_pool, int32_t num_slots, const int32_t* slot_idx,
                         int32_t* status, void* stream);

/* Selective scan: for every channel c with group g = c / (C / num_groups),
 *     dt = softplus(delta[t][c] + delta_bias[c])    (without softplus when delta_softplus is 0)
 *     h[n] = exp(dt * a[c][n]) * h[n] + dt * x[t][c] * b[t][g][n]
 *     y[t][c] = (sum_n c[t][g][n] * h[n] + d[c] * x[t][c]) * silu(z[t][c])
 * in fp32, y rounded once; states fp32 [C][state_dim]. */
typedef struct gdn_ssm_config {
  int32_t channels;        /* C, 1 .. 262,144, a multiple of num_groups */
  int32_t num_groups;
  int32_t state_dim;       /* N, 1 .. 128 */
  int32_t io_dtype;        /* gdn_dtype of x, delta, b, c, z and y */
  int32_t delta_softplus;
  const float* a;          /* [C][N] device (negative: decaying) */
  const float* d;          /* [C] device, or NULL: no skip term */
  const float* delta_bias; /* [C] device, or NULL */
} gdn_ssm_config;

/* The rows of a scan: row t of an array at its pointer + t * its stride (elements). x, delta, z
 * and y hold C elements a row (pointers 16-byte aligned, strides multiples of 16 bytes); b and c
 * [num_groups][N], at any alignment of their elements. z NULL: no gate. y may be x, delta or z
 * with the same stride; no other overlap. */
typedef struct gdn_ssm_rows {
  const void* x;
  const void* delta;
  const void* b;
  const void* c;
  const void* z;
  void* y;
  int64_t x_stride, delta_stride, b_stride, c_stride, z_stride, y_stride;
} gdn_ssm_rows;

/* Device workspace of gdn_ssm_packed for calls of at most these num_seqs, num_tokens and max_len
 * (multiple of 256; the host fields of req alone are read). */
gdn_status gdn_ssm_workspace_size(const gdn_ssm_config* cfg, const gdn_requests* req,
                                  size_t* bytes);

/* The scan of a pack of requests.
 *  state_pool  [num_slots][C][N] fp32, updated in place.
 *  ckpt_states [num_ckpt][C][N] fp32, or NULL without checkpoints.
 *  workspace   256-byte aligned; not to be used by other work before this call's has finished.
 * Where the call has too few channels and requests to fill the GPU, requests longer than a
 * segment (chosen from num_tokens, max_len, C and N, never from device values) are cut: a first
 * kernel finds each segment's end state from zeros and its decay, a second runs the segments
 * from the joined states; results then differ from the uncut ones by fp32 rounding. Those of calls that
 * are not cut do not depend on the pack around a request. The same call gives the same bits. Inputs
 * that are not finite spoil their own channel of their own request.
 * Errors: INVALID_ARGUMENT, UNSUPPORTED (state_dim above 128, channels, more requests or rows),
 * WORKSPACE_TOO_SMALL, CUDA. */
gdn_status gdn_ssm_packed(gdn_handle* handle, const gdn_ssm_config* cfg, const gdn_requests* req,
                          const gdn_ssm_rows* rows, float* state_pool, float* ckpt_states,
                          void* workspace, size_t workspace_bytes, int32_t* status,
                          void* stream);

/* One token of `batch` decoding requests (one kernel): row b with the state in slot slot_idx[b]
 * (device; below 0: the row is skipped; slots distinct), updated in place. */
gdn_status gdn_ssm_step(gdn_handle* handle, const gdn_ssm_config* cfg, int32_t batch,
                        const gdn_ssm_rows* rows, float* state_pool, int32_t num_slots,
                        const int32_t* slot_idx, int32_t* status, void* stream);

/* Root-mean-square norm of every head of every token, with the residual's addition in front and
 * a gate and an 8-bit output behind:
 *     s = x + residual                              (sum receives s rounded to io_dtype)
 *     v = s / sqrt(mean(s^2) + eps) * (weight + weight_offset) * silu(gate)
 *     y = v rounded to io_dtype; codes = v / scale rounded to e4m3
 * in fp32 from the unrounded s. A scale covers scale_group columns, or with 0 the token's whole
 * row: max|v| / 448 over its finite values, or with scale_pow2 the least power of two at least
 * that; 2^-100 at least. Infinities are held as the largest finite value; a NaN stays NaN. */
typedef struct gdn_norm_config {
  int32_t num_heads;     /* heads of a row, each normalised by itself (1: the row) */
  int32_t dim;           /* elements of a head: any with one head, else 64, 128 or 256 */
  int32_t io_dtype;      /* gdn_dtype of x, residual, sum, gate and y */
  int32_t scale_group;   /* 0, 32, 64 or 128 (dividing dim) */
  int32_t scale_pow2;
  float eps;             /* >= 0 */
  float weight_offset;   /* 1 where the model keeps weight - 1 */
  const float* weight;   /* [dim] device, or NULL: ones (and no offset) */
} gdn_norm_config;

/* The norm of num_tokens rows of num_heads * dim elements (at most 32,768), one kernel.
 *  residual, sum, gate  NULL where not wanted (sum needs residual). y NULL where codes are given.
 *          A call of no rows checks none of the arrays.
 *  codes   [num_tokens] rows of e4m3 at codes + t * codes_stride (bytes), with
 *  scales  [num_tokens][num_heads * dim / scale_group, or 1] fp32; or both NULL.
 * Pointers 16-byte aligned (scales 4), strides multiples of 16 bytes. sum and y may each be x,
 * residual or gate with the same stride (in place); no other overlap.
 * Errors: INVALID_ARGUMENT, UNSUPPORTED, CUDA. */
gdn_status gdn_rms_norm(gdn_handle* handle, const gdn_norm_config* cfg, int32_t num_tokens,
                        const void* x, int64_t x_stride, const void* residual,
                        int64_t residual_stride, void* sum, int64_t sum_stride, const void* gate,
                        int64_t gate_stride, void* y, int64_t y_stride, void* codes,
                        int64_t codes_stride, float* scales, void* stream);

/* Draw a token from every row of logits (one kernel). With l the row's logits, m their maximum
 * and w_i = exp((l_i - m) / temperature), tokens in the order of falling logits, equal ones by
 * rising index:
 *   top_k  > 0: the first top_k tokens are kept;
 *   top_p  < 1: of these the shortest beginning whose weight reaches top_p of theirs (the first
 *          token at least);
 *   min_p  > 0: of these the tokens with w_i >= min_p (values above 1 count as 1).
 * The token drawn is the first, by index, at which the kept tokens' weights sum to more than u
 * times their total; logprob is the logarithm of its share of that total. temperature 0: the
 * token of the maximum, lowest index first, logprob 0.
 *  logits       row r at logits + r * stride (elements), io_dtype, any alignment of elements.
 *  temperature, top_k, top_p, min_p  [num_rows] device, or NULL: 1, off, off, off.
 *  u            [num_rows] device, random numbers of [0, 1) (others count as the nearest).
 *  token        [num_rows] int32 out; logprob [num_rows] fp32 out, or NULL.
 * A logit of -inf or NaN is never drawn; where a row has +inf, those alone are drawn from. A row
 * without any other logit, or with a temperature below 0 or a NaN among its settings, gives token
 * -1 and logprob -inf and raises status (may be NULL) to GDN_ERR_INVALID_ARGUMENT.
 * Weights are fixed-point numbers of 2^-44 of the maximum's, right to 2^-28 of their own value
 * (or a unit), and their sums are exact: results depend on no order of additions, and the same
 * call gives the same bits. Supported: vocab 1 .. 262,144.
 * Errors: INVALID_ARGUMENT, UNSUPPORTED, CUDA. */
gdn_status gdn_sample(gdn_handle* handle, int32_t io_dtype, int32_t num_rows, int32_t vocab,
                      const void* logits, int64_t stride, const float* temperature,
                      const int32_t* top_k, const float* top_p, const float* min_p,
                      const float* u, int32_t* token, float* logprob, int32_t* status,
                      void* stream);

/* ---- host-side scheduling policy (no device work) ---------------------------------- */

/* Prefix-cache checkpoint position of a prompt of `len` tokens on a grid of `block`
 * tokens: the last multiple of `block` that is <= len, moved back one block when it falls
 * within the prompt's last `tail` tokens, so the prompt can stay in the pack (sparkinfer
 * v0.6.28, bullet on checkpoints in the last 16 tokens; there tail = 16). Returns the
 * position, or 0 when no checkpoint remains (len < block after the move). */
int32_t gdn_ckpt_position(int32_t len, int32_t block, int32_t tail);

/* Mixed-step prompt budget (sparkinfer v0.6.4 release notes, "What changed"): walk the
 * waiting prompts oldest first (index order), at most `max_prompts` of them, giving each
 * min(remaining_i, budget_left) tokens until `budget` tokens are used. take_out[i]
 * receives prompt i's share (0 for prompts not served). Returns the number of prompts
 * served, or -1 on invalid arguments. */
int32_t gdn_mixed_budget(int32_t num_waiting, const int32_t* remaining_host, int32_t budget,
                         int32_t max_prompts, int32_t* take_out_host);

#ifdef __cplusplus
}
#endif

#endif /* GDN_H_ */
