/*
 * symmoe.h -- C ABI of the zero-copy MoE dispatch -> expert -> combine path
 * over a flat symmetric heap, for one GB300 (sm_103a).
 *
 * Source of the operations: the AMD technical blog "MORI CCO: Next-Generation
 * Collective Communication Object for GPUs" --
 *   - section "What is MORI CCO?": every window sits at the same offset in
 *     every rank's slot, so a peer address is window base + peer * per-rank
 *     size + offset;
 *   - section "Zero-copy MoE dispatch -> expert -> combine": dispatch writes
 *     each token straight into the receive window ("disp_out") of the rank
 *     that owns its expert, the expert GEMM reads that window in place and
 *     writes its output into the combine staging window ("out_tok", the
 *     combine_in view), and combine gathers those rows back, weighted;
 *   - section "Mega-MoE: mega-kernel co-design with FlyDSL": dispatch, expert
 *     GEMM and combine fused into one kernel launch;
 *   - section "GEMM + all-to-all fusion": GEMM -> A2A and A2A -> GEMM on the
 *     same windows (sym_gemm_a2a, sym_a2a_gemm);
 * and the "MORI CCO Guide", sections "1. Concepts" (device communicator
 * passed by value into kernels) and "3. Memory and Windows" (collective
 * registration at identical offsets).
 *
 * Here the W "ranks" are W logical slots carved at identical offsets inside
 * ONE device allocation; a cross-slot store is a plain global store to
 * base + slot * per_rank_size + offset.
 *
 * Conventions for every call:
 *   - All pointers named dev_* or documented as device pointers must point to
 *     device memory of the current CUDA device; the library never allocates,
 *     frees or copies to/from host memory except in sym_heap_status (which
 *     reads one status word) -- the caller owns every buffer.  The library's
 *     own resources are a static device array (moe_dispatch_layout_noalloc)
 *     and, for sym_a2a_gemm's copy-engine form, two side streams and three
 *     events per device, created on first use and kept for the process.
 *   - bf16 tensors are passed as uint16_t bit patterns, row-major, contiguous.
 *   - All compute calls are asynchronous on `stream` (a cudaStream_t; NULL is
 *     the legacy default stream) and never synchronise the host.  Calls on
 *     one heap must run one after another on the GPU (one stream, or streams
 *     ordered by events): they share its windows and the work counters in
 *     its control window, which every launch leaves at zero when it ends.
 *   - Return value: SYM_OK (0) or a negative SYM_E* code, detected
 *     synchronously (bad argument, too small a heap, launch failure).
 *     Conditions found on the device while a kernel runs (a bounded wait that
 *     expired, a row beyond capacity) are OR-ed into the heap's status word
 *     and read with sym_heap_status; no kernel traps or aborts.
 *
 * Shapes (moe_shape): W = world slots, T = tokens per slot, N = W*T global
 * tokens (global token g = s*T + t lives on slot s), H = hidden, I = expert
 * intermediate size, E = experts, E/W experts per slot (expert e lives on
 * slot e / (E/W)), k = top-k.  Limits: E % W == 0, 1 <= k <= min(E, 32),
 * E <= 1024, H % 128 == 0, I % 128 == 0, H, I <= 65536.
 *
 * Accuracy: the expert FFN accumulates in fp32 on the tensor cores, whose
 * additions into the accumulator truncate.  Against an exact (fp64)
 * reference, bf16 outputs stay within 2e-2 * max(1, |ref|) per element and
 * 1e-2 relative L2 for K = H or I up to 16384 with weights ~N(0, 0.02).  At
 * K = 65536 with weights that large, |h| reaches ~200 and the truncation
 * over 4096 MMAs moves a few y elements in 10^4 just past that per-element
 * bound (relative L2 stays ~1e-3); the bound holds there for weights scaled
 * like a trained layer (about 1/sqrt(H): gate/up ~N(0, 0.0025) was checked).
 */
#ifndef SYMMOE_H
#define SYMMOE_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st *symmoe_stream_t; /* == cudaStream_t */

/* ---- status codes -------------------------------------------------------- */
#define SYM_OK 0
#define SYM_EINVAL (-1)    /* bad shape, pointer, alignment or argument        */
#define SYM_ENOSPACE (-2)  /* heap (or a window of it) too small for the call  */
#define SYM_ECUDA (-3)     /* a CUDA runtime call or kernel launch failed      */
#define SYM_ETIMEOUT (-4)  /* (status word) a bounded device wait expired      */
#define SYM_EOVERFLOW (-5) /* (status word) a row index beyond its window      */
#define SYM_ENOTSUP (-6)   /* not supported on this device (needs sm_103a)     */

/* bits of the device status word */
#define SYM_STATUS_TIMEOUT 0x1
#define SYM_STATUS_OVERFLOW 0x2

/* rows covered by one dispatch ready counter (per slot, per row block) */
#define SYM_ROWS_PER_FLAG 128
/* tokens per dispatch counting chunk */
#define SYM_COUNT_CHUNK 128

typedef struct moe_shape {
  int32_t world;           /* W */
  int32_t tokens_per_slot; /* T */
  int32_t hidden;          /* H */
  int32_t inter;           /* I */
  int32_t num_experts;     /* E */
  int32_t topk;            /* k */
} moe_shape;

/*
 * sym_heap: the symmetric heap descriptor.  Plain old data, passed BY VALUE
 * into every kernel (the device-communicator rule of the CCO guide).  Every
 * off_* is a byte offset inside EACH slot; window w of slot d is at
 * base + d * per_rank_size + off_w.  Per-slot windows:
 *   recv_x    [cap][H] bf16  dispatched token rows ("disp_out")
 *   y         [cap][H] bf16  expert outputs ("out_tok", combine_in view)
 *   h         [cap][I] bf16  SwiGLU intermediate of the expert FFN
 *   recv_pair [cap] int32    g*k + j of the pair that filled each row
 *   recv_w    [cap] fp32     routing weight of that pair
 *   pos       [T][k] int32   receive row of each of this slot's own pairs
 *                            (the "routing" handle combine uses)
 *   signal area: cnt [E/W] int32, recv_off [E/W] int32, total_recv int32,
 *                status int32 (slot 0's is the heap status word),
 *                ready [ceil(cap/128)] uint32 (rows landed per 128-row block)
 *   scratch (used in slot 0 only): dispatch chunk histograms, fused-kernel
 *                control block.
 * Every window is followed by a guard band of at least SYM_GUARD_BYTES that
 * no call reads or writes (sym_heap_windows gives each window's extent), so
 * a caller or a test can fill the bands with a pattern and check it after a
 * call.  Counts the kernels read back from the signal area are checked
 * against the window capacity: an expert whose rows [recv_off, recv_off +
 * cnt) or a slot whose total_recv do not fit in [0, cap) is skipped and
 * SYM_STATUS_OVERFLOW is raised (a corrupted or stale signal area never
 * sends a store past a window).
 * Receive rows are grouped by expert (ascending) inside a slot; inside one
 * expert they are in (source slot, token, k) order.
 */
#define SYM_GUARD_BYTES 1024
#define SYM_HEAP_WINDOWS 13
typedef struct sym_heap {
  uint64_t base;          /* device address of slot 0                          */
  uint64_t per_rank_size; /* slot stride in bytes (multiple of align)          */
  uint64_t bytes;         /* W * per_rank_size                                 */
  uint64_t cap;           /* receive rows per slot = N * min(k, E/W)           */
  uint64_t off_recv_x, off_y, off_h, off_recv_pair, off_recv_w, off_pos;
  uint64_t off_cnt, off_recv_off, off_total, off_status, off_ready;
  uint64_t off_hist;      /* chunk histograms, E * ceil(N/32) int32            */
  uint64_t off_ctrl;      /* fused-kernel counters and per-tile readiness      */
  uint32_t num_ready;     /* ready counters per slot = ceil(cap / 128)         */
  uint32_t epoch;         /* bumped by every dispatch / pipeline call          */
  uint32_t wait_timeout_us; /* bound on every device-side wait (default 2 s)   */
  uint32_t reserved;
  moe_shape s;
} sym_heap;

/*
 * sym_heap_bytes: size of the heap a shape needs.
 *   align: slot stride granularity in bytes (power of two >= 256; 0 = 2 MiB).
 *          align = 1<<32 reproduces the CCO kernel's 4 GiB-multiple stride.
 *   per_rank_size (out, may be NULL), total_bytes (out, may be NULL).
 * Host only.  Returns SYM_OK or SYM_EINVAL.
 */
int sym_heap_bytes(const moe_shape *s, uint64_t align, uint64_t *per_rank_size,
                   uint64_t *total_bytes);

/*
 * sym_heap_init: carve the windows into a caller-owned device allocation
 * (collective "alloc + register" of the CCO guide, reduced to arithmetic:
 * same windows, same order, same offsets in every slot).
 *   dev_base: device pointer, 256-byte aligned, owned by the caller, at least
 *             sym_heap_bytes(...) bytes, whose contents are zero before the
 *             first call that uses the heap (e.g. cudaMemsetAsync(dev_base, 0,
 *             bytes)): the status word and the fused-kernel counters start
 *             from zero.  The library keeps no reference other than the copy
 *             in *out.
 *   out:      filled descriptor (epoch 0, wait_timeout_us 2,000,000).
 * Host only, no device access.  SYM_EINVAL on a bad shape or alignment,
 * SYM_ENOSPACE if bytes is too small.
 */
int sym_heap_init(const moe_shape *s, void *dev_base, uint64_t bytes, uint64_t align,
                  sym_heap *out);

/*
 * sym_heap_slot_ptr: base + slot * per_rank_size + offset (the peer address
 * of "What is MORI CCO?").  Returns NULL if slot or offset is out of range.
 */
void *sym_heap_slot_ptr(const sym_heap *h, int slot, uint64_t offset);

/*
 * sym_heap_windows: the extent of every window inside a slot, in layout
 * order (recv_x, y, h, recv_pair, recv_w, pos, cnt, recv_off, total_recv,
 * status, ready, hist, ctrl): offsets[i] and bytes[i] for the first
 * min(max_windows, SYM_HEAP_WINDOWS) windows.  The bytes between the end of
 * window i and the start of window i + 1 (and after the last window, up to
 * per_rank_size) are the guard bands, at least SYM_GUARD_BYTES each.  Not in
 * the pages: a checking aid (a layout with guard bands stands in for a
 * memory checker).  Host only.  Returns SYM_HEAP_WINDOWS, or SYM_EINVAL.
 */
int sym_heap_windows(const sym_heap *h, uint64_t *offsets, uint64_t *bytes, int max_windows);

/*
 * moe_route_topk: per token, the top-k of E fp32 logits (descending, ties to
 * the lower expert index) and softmax weights over the selected k.
 *   logits: device [N][E] fp32;  idx: device [N][k] int32 (out);
 *   w: device [N][k] fp32 (out).  The pages leave routing to the caller; this
 *   is the router that feeds moe_dispatch.
 */
int moe_route_topk(const sym_heap *h, const float *logits, int32_t *idx, float *w,
                   symmoe_stream_t stream);

/*
 * moe_router_logits: the router (gate) GEMM that produces the routing logits
 * from the token activations (the step before moe_route_topk; the pages take
 * the routing as given):
 *   logits[g][e] = sum_h x[g][h] * w_router[e][h],  fp32 accumulation on the
 *   tensor cores, fp32 output.
 *   x: device [N][H] bf16 (16-byte aligned);  w_router: device [E][H] bf16
 *   (16-byte aligned);  logits: device [N][E] fp32.  N, H, E from the heap's
 *   shape.  When there are fewer output tiles than CTA pairs, K is split
 *   across pairs: the fp32 partials go to slot 0's y window (the expert
 *   output, which holds nothing between a combine and the next expert FFN)
 *   and a second kernel adds them in split order, so the logits do not depend
 *   on the schedule.  The call must therefore not overlap an expert FFN or a
 *   combine on the same heap; it writes nothing else of the heap but the
 *   status word.
 * Returns SYM_OK, SYM_EINVAL (pointer/alignment) or SYM_ECUDA; asynchronous.
 */
int moe_router_logits(const sym_heap *h, const uint16_t *x, const uint16_t *w_router, float *logits,
                      symmoe_stream_t stream);

/*
 * moe_router_splits: the number of K splits moe_router_logits uses for this
 * heap's shape on the current device (1: one GEMM launch writing the logits;
 * S > 1: S partials in slot 0's y window and one reduction launch).  No
 * device work; host only apart from reading the device's SM count.
 *   splits: host int (out).
 * Returns SYM_OK, SYM_EINVAL (bad heap or NULL splits) or SYM_ECUDA.
 */
int moe_router_splits(const sym_heap *h, int *splits);

/*
 * moe_dispatch: the all-to-all scatter of "Zero-copy MoE dispatch".
 * Counts pairs per expert, builds receive offsets, and copies every token row
 * x[g] into slot (idx[g][j] / (E/W))'s recv_x window at its receive row
 * (16-byte vector stores), writing recv_pair / recv_w / pos and raising the
 * ready counters (release) of the row blocks it fills.
 *   x: device [N][H] bf16;  idx, w: device [N][k] (from moe_route_topk or the
 *   caller; every idx must be in [0, E) and the k experts of a token distinct).
 *   Bumps h->epoch.  Out-of-range rows are skipped and flagged
 *   SYM_STATUS_OVERFLOW in the status word.
 */
int moe_dispatch(sym_heap *h, const uint16_t *x, const int32_t *idx, const float *w,
                 symmoe_stream_t stream);

/*
 * moe_dispatch_ex: moe_dispatch with flags.  SYM_DISPATCH_DEDUP: the
 * rank-deduplicated dispatch (a reading of "Zero-copy MoE dispatch" in which
 * a token crosses to each destination slot once): every token row is stored
 * once per distinct destination slot, into that slot's staging rows (its y
 * window, rows ordered by token g; the y window holds nothing until the down
 * GEMM), and each slot then expands its staged rows to its expert rows
 * locally.  The windows the expert FFN and the combine read (recv_x,
 * recv_pair, recv_w, pos, counts, offsets, ready counters) come out
 * bit-identical to moe_dispatch's.  Scratch in the h windows (idle until the
 * gate/up GEMM).  Needs W <= 32 and h windows of at least
 * 4*(cap + W*ceil(N/32) + N*k) bytes (cap*I*2; true for I >= 128 and k <= 32
 * but checked): SYM_EINVAL otherwise, or for an unknown flag.
 */
#define SYM_DISPATCH_DEDUP 1
/*
 * SYM_DISPATCH_FP8: the FP8 dispatch with per-token scales (the blog's
 * dispatch carries scales, recv_s).  Each row crosses as OCP E4M3 codes (H
 * bytes instead of 2H) with one scale 2^e per token, the smallest power of
 * two with max|x| <= 448 * 2^e (so x / 2^e is exact; the codes round to
 * nearest, ties to even).  The codes of pair row p land in row p of the
 * destination slot's y window (H bytes a row), the scale in word p of its h
 * window (fp32); the slot multiplies back to bf16 (exact) into recv_x.  The
 * expert FFN then sees the dequantized rows: results differ from the bf16
 * dispatch by the E4M3 rounding of x.  Not with SYM_DISPATCH_DEDUP.
 */
#define SYM_DISPATCH_FP8 2
int moe_dispatch_ex(sym_heap *h, const uint16_t *x, const int32_t *idx, const float *w, int flags,
                    symmoe_stream_t stream);

/*
 * moe_expert_ffn: expert_gemm of "Zero-copy MoE dispatch", here a SwiGLU FFN
 * per expert on its received rows, in place on the heap:
 *   h = bf16(silu(recv_x Wg_e^T) * (recv_x Wu_e^T)),  y = bf16(h Wd_e^T),
 * fp32 accumulation on the tensor cores (tcgen05, TMEM, TMA).  Row counts are
 * read on the device (no host sync); before loading a row block the kernel
 * waits (bounded) for its dispatch ready counter.
 *   w_gate, w_up: device [E][I][H] bf16;  w_down: device [E][H][I] bf16.
 * Writes the h and y windows of every slot.
 */
int moe_expert_ffn(const sym_heap *h, const uint16_t *w_gate, const uint16_t *w_up,
                   const uint16_t *w_down, symmoe_stream_t stream);

/*
 * moe_expert_ffn_ex: moe_expert_ffn with flags (0: identical to it).
 *   SYM_FFN_WEIGHTED_ROWS: the routing weights move from the combine into the
 *     expert epilogue (a variant; the pages apply them where combine takes
 *     them): y[p] = bf16(recv_w[p] * (h Wd_e^T)[p]), the weight of the row's
 *     (token, k) pair, written by moe_dispatch, multiplying the fp32
 *     accumulators before the one rounding.  Pair with moe_combine_ex and
 *     SYM_COMBINE_UNWEIGHTED.
 * Any other flag bit: SYM_EINVAL.
 */
#define SYM_FFN_WEIGHTED_ROWS 1
int moe_expert_ffn_ex(const sym_heap *h, const uint16_t *w_gate, const uint16_t *w_up,
                      const uint16_t *w_down, int flags, symmoe_stream_t stream);

/*
 * moe_combine: the weighted all-to-all gather of "Zero-copy MoE dispatch":
 *   out[g] = bf16( sum_{j<k} w[g][j] * y[slot(idx[g][j])][pos[g][j]] ),
 * fp32 accumulation in j order.
 *   expert_out: NULL or the address of slot 0's y window -> zero copy (the
 *     data_ptr match of the pages).  Any other device pointer is read as a
 *     dense [W][cap][H] bf16 tensor whose rows [0, total_recv[d]) are first
 *     copied into the y windows (the pages' silent fallback copy; counted by
 *     moe_combine_fallback_copies), with the identical result.
 *   idx, w: device [N][k] as given to moe_dispatch;  out: device [N][H] bf16.
 */
int moe_combine(const sym_heap *h, const uint16_t *expert_out, const int32_t *idx,
                const float *w, uint16_t *out, symmoe_stream_t stream);

/*
 * moe_combine_ex: moe_combine with flags (0: identical to it).
 *   SYM_COMBINE_UNWEIGHTED: the rows already carry their weights
 *     (SYM_FFN_WEIGHTED_ROWS): out[g] = bf16(sum_{j<k} y[slot(idx[g][j])][pos[g][j]]),
 *     fp32 sum in j order; w is not read and may be NULL.
 * Any other flag bit: SYM_EINVAL.
 */
#define SYM_COMBINE_UNWEIGHTED 1
int moe_combine_ex(const sym_heap *h, const uint16_t *expert_out, const int32_t *idx,
                   const float *w, uint16_t *out, int flags, symmoe_stream_t stream);

/* Number of fallback copies moe_combine has made in this process. */
uint64_t moe_combine_fallback_copies(void);

/*
 * moe_pipeline: route -> dispatch -> expert FFN -> combine on one stream.
 *   mode bits:
 *   SYM_PIPE_FUSED (1): one persistent launch ("Mega-MoE"): expert tiles start
 *     as soon as the ready counters of their rows land; without it one launch
 *     per stage (7 kernels).
 *   SYM_PIPE_WEIGHTS_IN_FFN (2): routing weights applied in the expert
 *     epilogue and an unweighted combine (SYM_FFN_WEIGHTED_ROWS,
 *     SYM_COMBINE_UNWEIGHTED).
 *   SYM_PIPE_DEDUP (4): the staged pipeline with the rank-deduplicated
 *     dispatch (moe_dispatch_ex, SYM_DISPATCH_DEDUP); not with SYM_PIPE_FUSED.
 *   SYM_PIPE_FP8 (8): the staged pipeline with the FP8 dispatch
 *     (SYM_DISPATCH_FP8); not with SYM_PIPE_FUSED or SYM_PIPE_DEDUP.
 *   Any other bit: SYM_EINVAL.  mode 0 / 1 are the staged / fused pipeline.
 *   idx, w: device [N][k] outputs of the routing step; out: device [N][H].
 *   Bumps h->epoch.
 */
#define SYM_PIPE_FUSED 1
#define SYM_PIPE_WEIGHTS_IN_FFN 2
#define SYM_PIPE_DEDUP 4
#define SYM_PIPE_FP8 8
int moe_pipeline(sym_heap *h, const float *logits, const uint16_t *x, const uint16_t *w_gate,
                 const uint16_t *w_up, const uint16_t *w_down, int32_t *idx, float *w,
                 uint16_t *out, int mode, symmoe_stream_t stream);

/*
 * sym_heap_status: synchronises `stream`, reads the heap status word (slot 0)
 * into *status (SYM_STATUS_* bits) and, if clear != 0, resets it to 0.
 * Returns SYM_OK, SYM_EINVAL or SYM_ECUDA.
 */
int sym_heap_status(const sym_heap *h, int32_t *status, int clear, symmoe_stream_t stream);

/*
 * GEMM + all-to-all fusion, a second workload on the same heap (blog,
 * "Examples", "GEMM + all-to-all fusion": GEMM -> A2A with the epilogue
 * writing output tiles straight into the peers' windows; A2A -> GEMM
 * consuming remote K-shards as they arrive, polling ready counters; each
 * against a split pipeline).  One linear layer w [H][H] (bf16, [out][in],
 * 16-byte aligned) is shared by the W slots; fp32 accumulation on the tensor
 * cores, bf16 results.  mode: SYM_LA_FUSED for the fused form, 0 for the split
 * pipeline (same results, bit for bit).  Neither call may overlap a
 * dispatch, expert FFN or combine on the same heap (they share its windows).
 */
#define SYM_LA_FUSED 1
#define SYM_LA_COPY_ENGINES 2 /* with SYM_LA_FUSED, sym_a2a_gemm only */

/*
 * sym_gemm_a2a: GEMM -> A2A.  Slot s computes Y_s = x_s w^T for its rows
 * x_s = x[s*T, (s+1)*T), and the rows are exchanged all-to-all in W blocks of
 * B = T/W rows: row s*B + r of slot j's y window receives Y_s[j*B + r].
 *   x: device [N][H] bf16, 16-byte aligned.
 *   fused: the GEMM epilogue stores each row at its destination;
 *   split: the GEMM stores Y_s in rows [0, T) of slot s's recv_x window, then
 *   a copy kernel exchanges the blocks.
 * Requires T % W == 0.  Writes rows [0, T) of every y window (split: also of
 * every recv_x window).  Returns SYM_OK, SYM_EINVAL or SYM_ECUDA; async.
 */
int sym_gemm_a2a(const sym_heap *h, const uint16_t *x, const uint16_t *w, int mode,
                 symmoe_stream_t stream);

/*
 * sym_a2a_gemm: A2A -> GEMM.  Slot s holds the K-shard s (features
 * [s*H/W, (s+1)*H/W)) of all N tokens: z [W][N][H/W] bf16, 16-byte aligned
 * (z[s] plays slot s's window).  Slot j computes C_j = U_j w^T into rows
 * [0, T) of its y window, U_j = its tokens j*T + r with every feature (shard s
 * at columns [s*H/W, (s+1)*H/W)).
 *   mode SYM_LA_FUSED: the all-to-all is the GEMM's operand loads: a tile of
 *   slot j reads K shard s of its tokens straight from z[s] (nothing copied).
 *   mode SYM_LA_FUSED | SYM_LA_COPY_ENGINES: slot j's recv_x window receives
 *   its shards shard major, [W][T][H/W], by one cudaMemcpyAsync per (slot,
 *   shard) on the copy engines from the library's side streams, each followed
 *   by a stream write of 1 into word s of slot j's ready window; the GEMM runs
 *   at the same time and its producer waits (bounded) for a shard's word
 *   before it loads that K range.  A wait that expires sets
 *   SYM_STATUS_TIMEOUT.  The call is ordered on `stream` as a whole.  Needs W
 *   words in a ready window (SYM_ENOSPACE if the heap has fewer).
 *   mode 0 (split): an SM copy kernel into the same shard-major blocks, then
 *   the GEMM.
 * Requires H % (64*W) == 0 (whole K blocks per shard).  Returns SYM_OK,
 * SYM_EINVAL, SYM_ENOSPACE or SYM_ECUDA; async.
 */
int sym_a2a_gemm(const sym_heap *h, const uint16_t *z, const uint16_t *w, int mode,
                 symmoe_stream_t stream);

/*
 * moe_dispatch_layout_noalloc: the dispatch layout without a heap, for
 * callers that cannot allocate device memory (a plug-in whose host framework
 * hands it only its input and output buffers and owns every allocation, or a
 * process that fixes its device-memory footprint at start-up).  The pages
 * have no counterpart: their dispatch always runs on a registered window.
 * Computes, from the routing indices alone, what moe_dispatch writes into the
 * heap's signal area and pos windows:
 *   idx:        device [N][k] int32, N = world * tokens_per_slot; every index
 *               in [0, E) and the k of a token distinct (an index outside
 *               [0, E) is not counted and gets pos -1; so does every later
 *               copy of an expert that a token lists twice, which is counted
 *               once);
 *   cnt:        device [E] int32 (out): pairs per expert;
 *   recv_off:   device [E] int32 (out): first receive row of each expert in
 *               its slot;
 *   total_recv: device [W] int32 (out): rows each slot receives;
 *   pos:        device [N][k] int32 (out): receive row of every pair in its
 *               destination slot, in the same order as moe_dispatch.
 * Only s->world, tokens_per_slot, num_experts and topk are used.
 * Scratch: a library-owned __device__ array of SYM_NOALLOC_HIST_MAX int32
 * (1 MiB, on every device that loads the library, until exit) holding the
 * E * ceil(N/128) chunk histograms; larger shapes return SYM_ENOSPACE.  The
 * call makes no device allocation.  Its first call on a device looks up the
 * array's address (cudaGetSymbolAddress) with that device current; make that
 * first call before any stream capture.  The address is kept per device and
 * looked up again on the first call after the device's context changed (after
 * cudaDeviceReset): that call, too, must come before any capture (under
 * capture it returns SYM_EINVAL).  All calls share the array: calls that
 * overlap on the GPU race on it and give wrong results.
 * Asynchronous on `stream`; SYM_OK, SYM_EINVAL, SYM_ENOSPACE or SYM_ECUDA.
 */
#define SYM_NOALLOC_HIST_MAX (1 << 18)
int moe_dispatch_layout_noalloc(const moe_shape *s, const int32_t *idx, int32_t *cnt,
                                int32_t *recv_off, int32_t *total_recv, int32_t *pos,
                                symmoe_stream_t stream);

/*
 * ---------------------------------------------------------------------------
 * Training through an MoE block.  The calls below work on plain tensors or on
 * a heap's windows alike (a sym_rows over a window); none needs a heap.  They
 * allocate nothing, keep no state between calls and may run on any streams at
 * the same time as long as their outputs (and workspaces) differ.
 *
 * Types: SYM_BF16, SYM_FP16 (the products), and SYM_FP32 (the other calls
 * too).  Sums, norms and products accumulate in 32 bits; every result is
 * rounded once, to its tensor's type.
 * ---------------------------------------------------------------------------
 */
#define SYM_BF16 0
#define SYM_FP16 1
#define SYM_FP32 2

/*
 * sym_rows: `slots` x `rows` rows of `cols` contiguous elements; row r of slot
 * d starts at element d * slot_stride + r * ld (slot_stride is not read when
 * slots == 1).  A plain [R][cols] tensor has slots = 1; the recv_x window of a
 * heap has slots = W, rows = cap, ld = H, slot_stride = per_rank_size / 2.
 */
typedef struct sym_rows {
  uint64_t ptr;
  int64_t ld;
  int64_t slot_stride;
  int64_t rows;
  int32_t slots;
  int32_t cols;
} sym_rows;

/*
 * sym_groups: the row ranges of the experts (groups).  Group e belongs to slot
 * d = e / (groups / slots) and owns rows [off, off + cnt) of it, with cnt =
 * cnt[d * cnt_slot_stride + e mod (groups / slots)] and off likewise, int32 in
 * device memory (read by the kernels; no host sync).  Ranges may leave gaps
 * but must not overlap.  A group whose range does not lie in [0, rows) of its
 * slot is taken as empty and SYM_STATUS_OVERFLOW is raised.
 *   status: device word that SYM_STATUS_* bits are OR-ed into, or NULL;
 *   wait_timeout_us: bound on each of the kernels' internal waits, for every output
 *   tile that it may span (0: 2,000,000); SYM_STATUS_TIMEOUT where one runs out.
 */
typedef struct sym_groups {
  const int32_t *cnt, *off;
  int64_t cnt_slot_stride, off_slot_stride;
  int32_t *status;
  int32_t groups;
  int32_t slots;
  uint32_t wait_timeout_us;
  uint32_t reserved;
} sym_groups;

/*
 * moe_grouped_matmul: the product of every group's rows with its own matrix:
 *   out[r][f] = sum_c x[r][c] * w[e][f][c]                     flags 0
 *   out[r][f] = sum_c x[r][c] * w[e][c][f]                     SYM_GM_TRANS_W
 * for the rows r of group e (F = out->cols, C = x->cols).  With w [E][F][C]
 * the first form is a linear layer's forward product and, on the same weights
 * with the sizes exchanged, the second its data gradient.
 *   dtype: SYM_BF16 or SYM_FP16, of x, w and out; accumulated in fp32 (few rows
 *   on the CUDA cores or by warp-wide products, more in tensor memory) in an order
 *   that depends on the sizes, the groups and the device's SM count, rounded once.
 *   w: device, 16-byte aligned; matrix e at element e * w_group_stride, its
 *   rows w_ld elements apart, both multiples of 8; matrices do not overlap.
 *   x: 16-byte aligned, ld (and slot_stride) multiples of 8.  out: any ld.
 *   slots, rows of x and out are equal.  Any C, F in [1, 65536], any number of
 *   rows per group; at most 1024 groups.
 * Rows of out outside every group are not written.  out must not overlap x
 * or w.  Returns SYM_OK, SYM_EINVAL or SYM_ECUDA; asynchronous.
 */
#define SYM_GM_TRANS_W 1
int moe_grouped_matmul(const sym_groups *g, int dtype, const sym_rows *x, const void *w,
                       int64_t w_group_stride, int64_t w_ld, int flags, const sym_rows *out,
                       symmoe_stream_t stream);

/*
 * moe_grouped_wgrad: the weight gradient of moe_grouped_matmul,
 *   dw[e][f][c] = sum over the rows r of group e of dy[r][f] * x[r][c],
 * zeros for a group without rows.  SYM_GM_ACCUMULATE: added to what dw holds
 * (a group without rows is left as it is).
 *   dtype: SYM_BF16 or SYM_FP16, of dy and x; out_dtype: that, or SYM_FP32.
 *   dy, x: as x above, equal slots and rows.  dw: device; matrix e at element
 *   e * dw_group_stride, its rows dw_ld elements apart (any strides; 16-byte
 *   aligned ones are stored faster).
 * The contraction runs over the group's rows in order, one work item per
 * output tile: the result does not depend on the schedule.  The tensor
 * cores' additions into the fp32 accumulator truncate: an fp32 result is off by
 * about 1e-9 of its norm for every row of the group (measured relative L2: 2.3e-7
 * at 256 rows, 1.0e-6 at 1024, 4.4e-6 at 4096), far below a 16-bit result's
 * rounding (2e-3).
 */
#define SYM_GM_ACCUMULATE 1
int moe_grouped_wgrad(const sym_groups *g, int dtype, const sym_rows *dy, const sym_rows *x,
                      void *dw, int64_t dw_group_stride, int64_t dw_ld, int out_dtype, int flags,
                      symmoe_stream_t stream);

/*
 * moe_swiglu_rows: what stands between the grouped products of a SwiGLU
 * expert, h = row_w * silu(g) * u per row, with the row's routing weight (or
 * 1): with the weight here, the combine that follows is the unweighted one and
 * the weight's gradient a sum over the row.
 *   dtype: SYM_BF16, SYM_FP16 or SYM_FP32, of g, u and h (equal slots, rows,
 *   cols; any strides: rows that all start at the same place of a 16-byte line
 *   in every tensor move in 16-byte vectors).
 *   row_w: device fp32, row r of slot d at d * row_w_slot_stride + r; or NULL.
 *   total: device int32, total[d * total_slot_stride] = rows of slot d to do
 *   (read by the kernel, cut to [0, rows]); NULL: all.  Other rows are not
 *   read or written.
 * The exponential is the fast one for every type: silu is off by 2e-7 relative
 * for positive g, 1e-6 at g = -20 and 2e-6 at -30 (the norms' sigmoid gates too).
 * h may be g or u.  Returns SYM_OK, SYM_EINVAL or SYM_ECUDA; asynchronous.
 */
int moe_swiglu_rows(int dtype, const sym_rows *g, const sym_rows *u, const float *row_w,
                    int64_t row_w_slot_stride, const int32_t *total, int64_t total_slot_stride,
                    const sym_rows *h, symmoe_stream_t stream);

/*
 * moe_swiglu_rows_bwd: the gradients of moe_swiglu_rows from dh:
 *   dg = row_w * dh * u * silu'(g),  du = row_w * dh * silu(g),
 *   d_row_w[r] = sum_c dh * silu(g) * u   (fp32, strided like row_w; or NULL).
 * dg may be g or dh, du may be u.
 */
int moe_swiglu_rows_bwd(int dtype, const sym_rows *g, const sym_rows *u, const sym_rows *dh,
                        const float *row_w, int64_t row_w_slot_stride, const int32_t *total,
                        int64_t total_slot_stride, const sym_rows *dg, const sym_rows *du,
                        float *d_row_w, int64_t d_row_w_slot_stride, symmoe_stream_t stream);

/*
 * moe_dropout: y = residual + x * keep / (1 - p) (residual may be NULL), where
 * the element with index i = (slot * rows + row) * cols + column is kept iff
 * word(i) >= floor(p * 2^32).  word(i) is word i mod 4 of block i / 4 of
 * Philox 4x32-10 under the key `seed` and the upper counter half `offset`: the
 * mask is a function of (seed, offset, i) and never stored; the same call on
 * the output's gradient is the backward pass.  A dropped element contributes
 * exactly 0, whatever x holds there (infinities and NaN too).
 *   dtype: SYM_BF16, SYM_FP16 or SYM_FP32.  0 <= p < 1.
 * y may be x or residual.  Returns SYM_OK, SYM_EINVAL or SYM_ECUDA; async.
 */
int moe_dropout(int dtype, const sym_rows *x, const sym_rows *residual, const sym_rows *y,
                double p, uint64_t seed, uint64_t offset, symmoe_stream_t stream);

/*
 * moe_block_norm: the norms before and after a block in one pass over the
 * rows, with the block's gate, dropout and residual scale:
 *   n = o * rstd_post * w_post       rstd_post = 1 / sqrt(mean(o^2) + eps)
 *   y = x + scale * drop(act(gate) * n)
 *   h = y * rstd_pre * w_pre         rstd_pre = 1 / sqrt(mean(y^2) + eps)
 * o: the block's output; x: the residual stream; y: the stream after the
 * block; h: the next block's input, from the unrounded y.
 *   o NULL: the norm before a first block only (y = x; y is not written).
 *   SYM_NORM_NO_POST: no norm after the block (n = o; w_post, rstd_post NULL).
 *   h NULL: no norm before a next one.
 *   w_post, w_pre [cols]: NULL = ones.  gate [gate_rows][cols], row r uses gate
 *   row r / (rows / gate_rows): one gate for all rows, one for each sequence
 *   or one for each row; NULL = ones.  gate_act: SYM_GATE_*.
 *   p, seed, offset: dropout as in moe_dropout, element index row * cols + col.
 *   (A dropped element passes nothing on, whatever it holds, forward or backward;
 *   the norm after the block takes rstd_post from all of o's row, though.)
 *   rstd_post, rstd_pre: device fp32 [rows], out (kept for the backward), each
 *   may be NULL.
 * All tensors have the type dtype; rows ld_* elements apart; vectors of 16
 * bytes are used when every base, stride and cols allow.  y may be x.
 * cols <= 65536; gate_rows divides rows; 0 <= p < 1; eps >= 0.
 */
#define SYM_GATE_NONE 0
#define SYM_GATE_SIGMOID 1
#define SYM_GATE_TANH 2
#define SYM_NORM_NO_POST 1
typedef struct sym_block_norm {
  int64_t rows;
  int32_t cols, dtype;
  const void *x, *o, *w_post, *gate, *w_pre;
  void *y, *h;
  float *rstd_post, *rstd_pre;
  int64_t ld_x, ld_o, ld_gate, ld_y, ld_h;
  int64_t gate_rows;
  int32_t gate_act, flags;
  float scale, eps;
  double p;
  uint64_t seed, offset;
} sym_block_norm;
int moe_block_norm(const sym_block_norm *a, symmoe_stream_t stream);

/*
 * moe_block_norm_bwd: gradients of moe_block_norm.  Of `a` it reads o, w_post,
 * gate, w_pre, y (the stream after the block; with o NULL the stream itself)
 * and rstd_post, rstd_pre as the forward left them; x, h and eps are not used.
 *   dy: gradient of y from elsewhere (NULL: none); dh: gradient of h (NULL:
 *   none; then y, w_pre, rstd_pre are not read).
 *   dx: gradient of x (= of y; may be dy); d_o, dw_pre, dw_post, dgate: each
 *   of the type of what it is the gradient of, each may be NULL.
 *   work: device, 16-byte aligned, at least moe_block_norm_workspace(...)
 *   bytes; contents do not matter before or after.
 * Column sums are taken in 32 bits in an order that depends on the sizes, the
 * type, on whether every base, stride and cols allow 16-byte vectors, and on the
 * device's SM count only.
 */
typedef struct sym_block_norm_grad {
  const void *dy, *dh;
  void *dx, *d_o, *dw_pre, *dw_post, *dgate;
  int64_t ld_dy, ld_dh, ld_dx, ld_do, ld_dgate;
  void *work;
  uint64_t work_bytes;
} sym_block_norm_grad;
int moe_block_norm_bwd(const sym_block_norm *a, const sym_block_norm_grad *g, symmoe_stream_t stream);

/* Workspace bytes of moe_block_norm_bwd (gate_rows 0: no gate gradient).  Host only. */
int moe_block_norm_workspace(int64_t rows, int32_t cols, int64_t gate_rows, uint64_t *bytes);

/*
 * moe_layer_norm: layer norm of rows, with the residual sum in the same pass:
 *   s = x + add                      (add NULL: s = x)
 *   h = (s - mean) * rstd * w + b    mean, rstd = 1 / sqrt(mean((s - mean)^2) + eps) of the row
 *   sum, if not NULL: s, rounded; h and the statistics come from the unrounded s.
 *   w, b [cols]: NULL = ones, zeros.  mean, rstd: device fp32 [rows], out (kept
 *   for the backward), each may be NULL.  h may be NULL.
 * All tensors have the type dtype; rows ld_* elements apart; 16-byte vectors are
 * used where a row starts on a 16-byte boundary in every tensor, or equally far from
 * one (what lies between a tensor's rows may then be read, and is not used).  h or sum
 * may be x or add, but sum is not h.
 * The variance is the mean of the squared distances from the mean, all in fp32.
 * rows < 2^30, cols <= 65536; eps >= 0; |s| up to 1.7e38 (half of fp32's range: distances
 * from the mean are taken in it).  A row whose s holds an infinity or NaN, and only that
 * row, has an rstd and an h of NaN (its mean is what its sum gives).
 */
typedef struct sym_layer_norm {
  int64_t rows;
  int32_t cols, dtype;
  const void *x, *add, *w, *b;
  void *sum, *h;
  float *mean, *rstd;
  int64_t ld_x, ld_add, ld_sum, ld_h;
  float eps;
  uint32_t reserved;
} sym_layer_norm;
int moe_layer_norm(const sym_layer_norm *a, symmoe_stream_t stream);

/*
 * moe_layer_norm_bwd: gradients of moe_layer_norm, n = (s - mean) * rstd:
 *   g = dh * w;   dx = dsum + rstd * (g - mean(g) - n * mean(g * n))
 *   dw = sum over the rows of dh * n,   db = sum over the rows of dh.
 *   s: the forward's s (x, or sum where something was added); mean, rstd as the
 *   forward left them; dsum: gradient of s from elsewhere, or NULL.
 *   dx is the gradient of x and of add; may be dh, dsum or s.  dx, dw, db: each may be NULL.
 *   work: device, 16-byte aligned, at least moe_layer_norm_workspace(...) bytes;
 *   contents do not matter before or after; not read where dw and db are NULL.
 * The column sums are taken in 32 bits in an order that depends on the sizes, the
 * type, the alignment and the device's SM count only.
 */
typedef struct sym_layer_norm_grad {
  int64_t rows;
  int32_t cols, dtype;
  const void *dh, *s, *dsum, *w;
  const float *mean, *rstd;
  void *dx, *dw, *db;
  int64_t ld_dh, ld_s, ld_dsum, ld_dx;
  void *work;
  uint64_t work_bytes;
} sym_layer_norm_grad;
int moe_layer_norm_bwd(const sym_layer_norm_grad *a, symmoe_stream_t stream);

/* Workspace bytes of moe_layer_norm_bwd.  Host only. */
int moe_layer_norm_workspace(int64_t rows, int32_t cols, uint64_t *bytes);

/*
 * moe_orthogonalize: a batch of updates with their singular values brought
 * towards one by Newton-Schulz products (the experts' weight gradients of
 * moe_grouped_wgrad, or momentum made of them):
 *   X = g / (|g| + eps)              |g|: the square root of the sum of squares of a matrix
 *   `steps` times   X = a X + (b A + c A A) X,  A = X X^T    (rows <= cols;
 *                   X = a X + X (b A + c A A),  A = X^T X     otherwise: the same X)
 *   out = scale * X
 * with (a, b, c) = coeffs.  A matrix of zeros gives zeros; one that holds an
 * infinity or NaN, and only that one, gives NaN.
 *   g: device, count matrices of rows x cols, matrix i at element i * g_stride,
 *   its rows ld_g elements apart, of type g_dtype (SYM_BF16, SYM_FP16, SYM_FP32).
 *   out: likewise, of type out_dtype (SYM_BF16 or SYM_FP16); may be g where type
 *   and strides are equal.
 *   Any strides; rows, cols in [1, 65536], count in [0, 65535], steps in [0, 64].
 *   work: device, 256-byte aligned.  moe_orthogonalize_workspace gives what lets
 *   all matrices go side by side where they are small, and enough of them at a
 *   time to fill the device where they are large (work_bytes), and the least the
 *   call takes (least_bytes): the matrices go through in as many turns as the
 *   workspace makes them.  Contents do not matter before or after.  (Products are cut
 *   up by the number of matrices in a turn: another one can change last bits.)
 *   status: device word that SYM_STATUS_TIMEOUT is OR-ed into where one of the
 *   products' internal waits runs out (wait_timeout_us each, 0: 2,000,000), or NULL.  Out is
 *   undefined then, and nothing else tells of it.
 * X is held in 22 bits (two fp16 numbers); a Gram matrix and its polynomial are held as
 * their diagonals in fp32 and the rest in fp16; products accumulate in fp32 on the tensor
 * cores.  Products take 11 bits of an operand, and 22 (of X, and of the Gram matrices' rest) in
 * all steps for fp16 results and in all but the last two for matrices with a side of 512 or less.
 * Against exact arithmetic, five steps with (3.4445, -4.7750, 2.0315) are off, before the
 * result's rounding (1.7e-3 of its norm in bf16, 2.1e-4 in fp16), by
 *   fp16 results: 2e-4 of the norm; gradients of a few directions with next to nothing (1e-3
 *   or less) beside them, where errors grow 480 times in five steps, 6e-4 (with a shorter
 *   side above 2048 in proportion to it);
 *   bf16 results: 3e-4 to 6e-4, where a gradient has a few directions alone or few
 *   elements 1.2e-3; matrices with a side below 16 up to 2e-3.
 * This holds whatever g's scale, as long as |g| is not far below eps and the coefficients
 * keep the singular values of X below 3.
 */
typedef struct sym_orthogonalize {
  int32_t count, rows, cols, steps;
  int32_t g_dtype, out_dtype;
  float coeffs[3];
  float eps, scale;
  uint32_t wait_timeout_us;
  int32_t *status;
  const void *g;
  void *out;
  int64_t g_stride, ld_g, out_stride, ld_out;
  void *work;
  uint64_t work_bytes;
} sym_orthogonalize;
int moe_orthogonalize(const sym_orthogonalize *a, symmoe_stream_t stream);
int moe_orthogonalize_workspace(int32_t count, int32_t rows, int32_t cols, uint64_t *work_bytes,
                                uint64_t *least_bytes);

/*
 * moe_few_tokens: a whole MoE layer for a few tokens (what a decode step of a
 * few users asks of it), without a heap, in two launches (three with the router):
 *   logits[t] = w_router x[t]                     (w_router NULL: logits are given)
 *   idx[t], w[t]: the top-k of the logits (descending, equal ones to the lower
 *   expert) and the softmax over them
 *   out[t] = sum_j w[t][j] * (silu(x Wg^T) * (x Wu^T)) Wd^T   of expert idx[t][j]
 * A chosen expert whose logit is -infinity has the weight 0 and takes no part; a
 * token without any other has a row of zeros.  A logit that is NaN ranks below
 * all numbers; where one is chosen, or +infinity is, the token's weights and row
 * are NaN.
 *   dtype: SYM_BF16 or SYM_FP16, of x, the weights and out.
 *   x [tokens][hidden], 16-byte aligned, ld_x a multiple of 8; may be out.
 *   logits [tokens][num_experts] fp32 (in, or out with w_router); idx int32, w fp32
 *   [tokens][topk] (out).
 *   w_gate, w_up: [num_experts][inter][hidden], w_down: [num_experts][hidden][inter],
 *   w_router: [num_experts][hidden]: 16-byte aligned, expert e at element
 *   e * *_group, rows *_ld elements apart (multiples of 8), so that w_gate and w_up
 *   may be the halves of one tensor.
 *   work: device, 16-byte aligned, moe_few_tokens_workspace(...) bytes; contents do
 *   not matter before or after.
 * tokens in [0, 32], hidden and inter multiples of 8 up to 65536, num_experts <= 1024,
 * topk <= min(num_experts, 32).  Products accumulate in fp32; h is held in two
 * numbers of dtype (bf16: 16 bits; fp16: 22, or to 2^-36 where it is below 2^-14, and
 * infinite beyond its range); out is rounded once.  Only the chosen experts' weights are read.
 */
typedef struct sym_few_tokens {
  int32_t tokens, hidden, inter, num_experts, topk, dtype;
  const void *x, *w_gate, *w_up, *w_down, *w_router;
  float *logits;
  int32_t *idx;
  float *w;
  void *out;
  int64_t ld_x, ld_out, gate_group, gate_ld, up_group, up_ld, down_group, down_ld, router_ld;
  void *work;
  uint64_t work_bytes;
} sym_few_tokens;
int moe_few_tokens(const sym_few_tokens *a, symmoe_stream_t stream);

/* Workspace bytes of moe_few_tokens.  Host only. */
int moe_few_tokens_workspace(int32_t tokens, int32_t inter, int32_t topk, uint64_t *bytes);

/* Static description of a SYM_* code (never NULL). */
const char *sym_strerror(int code);

#ifdef __cplusplus
}
#endif

#endif /* SYMMOE_H */
