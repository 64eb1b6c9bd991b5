// capi.cu -- the extern "C" boundary of libsymmoe: argument validation, the
// symmetric heap layout, and the launch sequence of every call.
//
// Heap layout (MORI CCO guide, "3. Memory and Windows": windows are registered
// collectively, in the same order and with the same size on every rank, so
// each sits at the same offset in every slot).  Windows of one slot, in this
// order, each 1024-byte aligned and followed by a guard band of at least
// SYM_GUARD_BYTES: recv_x, y, h, recv_pair, recv_w, pos, cnt, recv_off, total,
// status, ready, hist, ctrl.  per_rank_size is the sum rounded up to the
// caller's alignment.
#include <atomic>
#include <cstring>

#include "symmoe_dev.cuh"

namespace symmoe {
cudaError_t launch_route_topk(const sym_heap &h, const float *logits, int32_t *idx, float *w,
                              cudaStream_t st);
cudaError_t launch_dispatch(const sym_heap &h, const uint16_t *x, const int32_t *idx,
                            const float *w, int mode, cudaStream_t st);
cudaError_t launch_expert_ffn(const sym_heap &h, const uint16_t *wg, const uint16_t *wu,
                              const uint16_t *wd, int num_sms, int wait_ready, int scale_rows,
                              cudaStream_t st);
cudaError_t launch_combine(const sym_heap &h, const uint16_t *expert_out, const int32_t *idx,
                           const float *w, uint16_t *out, int unit_weights, int num_sms, cudaStream_t st);
cudaError_t launch_router(const sym_heap &h, const uint16_t *x, const uint16_t *wr, float *logits,
                          int num_sms, cudaStream_t st);
cudaError_t router_plan(const sym_heap &h, int num_sms, int *grid, int *splits, int *kb_per_split);
cudaError_t launch_gemm_a2a(const sym_heap &h, const uint16_t *x, const uint16_t *w, int fused, int num_sms,
                            cudaStream_t st);
cudaError_t launch_a2a_gemm(const sym_heap &h, const uint16_t *z, const uint16_t *w, int mode, int num_sms,
                            cudaStream_t st);
int a2a_gemm_counters(const sym_heap &h);
size_t fused_ctrl_bytes(const moe_shape &s);
cudaError_t launch_fused(const sym_heap &h, const float *logits, const uint16_t *x,
                         const uint16_t *wg, const uint16_t *wu, const uint16_t *wd,
                         int32_t *idx, float *w, uint16_t *out, int weights_in_ffn, int num_sms,
                         cudaStream_t st);
cudaError_t launch_grouped_matmul(const sym_groups &g, int fp16, const sym_rows &x, const void *w, int64_t w_group,
                                  int64_t w_ld, int trans, const sym_rows &out, int num_sms, cudaStream_t st);
bool few_rows_product(const sym_groups &g, const sym_rows &x, int trans);
cudaError_t launch_few_rows(const sym_groups &g, int fp16, const sym_rows &x, const void *w, int64_t w_group,
                            int64_t w_ld, int trans, const sym_rows &out, int num_sms, cudaStream_t st);
bool thin_product(const sym_groups &g, const sym_rows &x, const sym_rows &out, int trans, int num_sms);
cudaError_t launch_thin_product(const sym_groups &g, int fp16, const sym_rows &x, const void *w, int64_t w_group,
                                int64_t w_ld, int trans, const sym_rows &out, int num_sms, cudaStream_t st);
cudaError_t launch_grouped_wgrad(const sym_groups &g, int fp16, const sym_rows &dy, const sym_rows &x, void *dw,
                                 int64_t dw_group, int64_t dw_ld, int out_type, int add, int num_sms,
                                 cudaStream_t st);
cudaError_t launch_swiglu_rows(int dtype, const sym_rows &g, const sym_rows &u, const sym_rows &h, const float *rw,
                               int64_t rw_slot, const int32_t *total, int64_t total_slot, int num_sms,
                               cudaStream_t st);
cudaError_t launch_swiglu_rows_bwd(int dtype, const sym_rows &g, const sym_rows &u, const sym_rows &dh,
                                   const sym_rows &dg, const sym_rows &du, const float *rw, int64_t rw_slot,
                                   float *drw, int64_t drw_slot, const int32_t *total, int64_t total_slot,
                                   int num_sms, cudaStream_t st);
cudaError_t launch_dropout(int dtype, const sym_rows &x, const sym_rows *res, const sym_rows &y, uint64_t seed,
                           uint64_t offset, double drop, int num_sms, cudaStream_t st);
size_t block_norm_workspace(int64_t rows, int cols, int64_t gates, int num_sms);
cudaError_t launch_block_norm(const sym_block_norm &a, int num_sms, cudaStream_t st);
size_t layer_norm_workspace(int64_t rows, int cols, int num_sms);
cudaError_t launch_layer_norm(const sym_layer_norm &a, int num_sms, cudaStream_t st);
cudaError_t launch_layer_norm_bwd(const sym_layer_norm_grad &a, int num_sms, cudaStream_t st);
void orthogonalize_workspace(int count, int rows, int cols, int num_sms, size_t *least, size_t *best);
cudaError_t launch_orthogonalize(const sym_orthogonalize &a, int num_sms, cudaStream_t st);
size_t few_tokens_workspace(int tokens, int inter, int topk);
cudaError_t launch_few_tokens(const sym_few_tokens &a, int num_sms, cudaStream_t st);
cudaError_t launch_block_norm_bwd(const sym_block_norm &a, const sym_block_norm_grad &b, int num_sms,
                                  cudaStream_t st);
}  // namespace symmoe

using namespace symmoe;

namespace {

constexpr uint64_t kWinAlign = 1024;
constexpr uint64_t kDefaultAlign = 2ull << 20;
constexpr uint32_t kDefaultTimeoutUs = 2000000u;

std::atomic<uint64_t> g_fallback_copies{0};

uint64_t round_up(uint64_t v, uint64_t a) { return (v + a - 1) / a * a; }

bool shape_ok(const moe_shape *s) {
  if (!s) return false;
  const int64_t W = s->world, T = s->tokens_per_slot, H = s->hidden, I = s->inter,
                E = s->num_experts, k = s->topk;
  if (W < 1 || T < 1 || E < 1 || k < 1) return false;
  if (E % W != 0 || E > 1024) return false;
  if (k > E || k > 32) return false;
  if (H < 128 || H % 128 != 0 || H > 65536) return false;
  if (I < 128 || I % 128 != 0 || I > 65536) return false;
  const int64_t N = W * T;
  if (N * k >= (int64_t(1) << 31) || N >= (int64_t(1) << 31)) return false;
  return true;
}

struct Layout {
  uint64_t cap, off_recv_x, off_y, off_h, off_recv_pair, off_recv_w, off_pos, off_cnt,
      off_recv_off, off_total, off_status, off_ready, off_hist, off_ctrl, used;
  uint32_t num_ready;
  uint64_t win_off[SYM_HEAP_WINDOWS], win_bytes[SYM_HEAP_WINDOWS];  // in slot order
};

Layout layout_of(const moe_shape *s) {
  Layout L{};
  const uint64_t W = s->world, T = s->tokens_per_slot, H = s->hidden, I = s->inter,
                 E = s->num_experts, k = s->topk;
  const uint64_t N = W * T, E_loc = E / W;
  L.cap = N * (k < E_loc ? k : E_loc);
  L.num_ready = (uint32_t)((L.cap + SYM_ROWS_PER_FLAG - 1) / SYM_ROWS_PER_FLAG);
  uint64_t o = 0;
  int nwin = 0;
  // every window is followed by at least SYM_GUARD_BYTES that no call reads
  // or writes (a guard band: a store past a window's end lands there first)
  auto take = [&](uint64_t bytes) {
    const uint64_t at = o;
    L.win_off[nwin] = at;
    L.win_bytes[nwin++] = bytes;
    o = round_up(o + bytes + SYM_GUARD_BYTES, kWinAlign);
    return at;
  };
  L.off_recv_x = take(L.cap * H * 2);
  L.off_y = take(L.cap * H * 2);
  L.off_h = take(L.cap * I * 2);
  L.off_recv_pair = take(L.cap * 4);
  L.off_recv_w = take(L.cap * 4);
  L.off_pos = take(T * k * 4);
  L.off_cnt = take(E_loc * 4);
  L.off_recv_off = take(E_loc * 4);
  L.off_total = take(4);
  L.off_status = take(4);
  L.off_ready = take((uint64_t)L.num_ready * 4);
  // chunk histograms: 128-token chunks for the stand-alone dispatch, 32-token
  // chunks for the fused pipeline (the larger of the two)
  L.off_hist = take(E * ((N + 31) / 32) * 4);
  L.off_ctrl = take(fused_ctrl_bytes(*s));
  L.used = o;
  return L;
}

bool heap_ok(const sym_heap *h) {
  if (!h || !shape_ok(&h->s) || h->base == 0 || (h->base & 255u)) return false;
  const Layout L = layout_of(&h->s);
  return h->cap == L.cap && h->per_rank_size >= L.used && h->off_ctrl == L.off_ctrl &&
         h->num_ready == L.num_ready;
}

bool aligned16(const void *p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void *p) { return p && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// A host thread that has made no CUDA call yet has no current context, and the
// tensor-map encoder (a driver call) refuses without one: make the device's
// primary context current there.  A context the caller chose stays.
bool have_context(int dev) {
  typedef CUresult (*Fn)(CUcontext *);
  static const Fn current = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &p, 12000, cudaEnableDefault, &q);
    return e == cudaSuccess && q == cudaDriverEntryPointSuccess ? reinterpret_cast<Fn>(p) : nullptr;
  }();
  CUcontext c = nullptr;
  if (current && current(&c) == CUDA_SUCCESS && c) return true;
  return cudaSetDevice(dev) == cudaSuccess;
}

int num_sms_of_current_device() {
  static int cache[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || !have_context(dev)) return 0;
  if (dev < 64 && cache[dev]) return cache[dev];
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (dev < 64) cache[dev] = n;
  return n;
}

int from_cuda(cudaError_t e) { return e == cudaSuccess ? SYM_OK : SYM_ECUDA; }

}  // namespace

extern "C" {

int sym_heap_bytes(const moe_shape *s, uint64_t align, uint64_t *per_rank_size,
                   uint64_t *total_bytes) {
  if (!shape_ok(s)) return SYM_EINVAL;
  if (align == 0) align = kDefaultAlign;
  if (align < 256 || (align & (align - 1))) return SYM_EINVAL;
  const Layout L = layout_of(s);
  const uint64_t prs = round_up(L.used, align);
  if (per_rank_size) *per_rank_size = prs;
  if (total_bytes) *total_bytes = prs * (uint64_t)s->world;
  return SYM_OK;
}

int sym_heap_init(const moe_shape *s, void *dev_base, uint64_t bytes, uint64_t align,
                  sym_heap *out) {
  if (!out || !dev_base || (reinterpret_cast<uintptr_t>(dev_base) & 255u)) return SYM_EINVAL;
  uint64_t prs = 0, total = 0;
  const int rc = sym_heap_bytes(s, align, &prs, &total);
  if (rc != SYM_OK) return rc;
  if (bytes < total) return SYM_ENOSPACE;
  const Layout L = layout_of(s);
  sym_heap h;
  std::memset(&h, 0, sizeof(h));
  h.base = reinterpret_cast<uint64_t>(dev_base);
  h.per_rank_size = prs;
  h.bytes = total;
  h.cap = L.cap;
  h.off_recv_x = L.off_recv_x;
  h.off_y = L.off_y;
  h.off_h = L.off_h;
  h.off_recv_pair = L.off_recv_pair;
  h.off_recv_w = L.off_recv_w;
  h.off_pos = L.off_pos;
  h.off_cnt = L.off_cnt;
  h.off_recv_off = L.off_recv_off;
  h.off_total = L.off_total;
  h.off_status = L.off_status;
  h.off_ready = L.off_ready;
  h.off_hist = L.off_hist;
  h.off_ctrl = L.off_ctrl;
  h.num_ready = L.num_ready;
  h.epoch = 0;
  h.wait_timeout_us = kDefaultTimeoutUs;
  h.s = *s;
  *out = h;
  return SYM_OK;
}

int sym_heap_windows(const sym_heap *h, uint64_t *offsets, uint64_t *bytes, int max_windows) {
  if (!heap_ok(h) || max_windows < 0 || (max_windows > 0 && (!offsets || !bytes))) return SYM_EINVAL;
  const Layout L = layout_of(&h->s);
  for (int i = 0; i < SYM_HEAP_WINDOWS && i < max_windows; ++i) {
    offsets[i] = L.win_off[i];
    bytes[i] = L.win_bytes[i];
  }
  return SYM_HEAP_WINDOWS;
}

void *sym_heap_slot_ptr(const sym_heap *h, int slot, uint64_t offset) {
  if (!h || slot < 0 || slot >= h->s.world || offset >= h->per_rank_size) return nullptr;
  return reinterpret_cast<void *>(h->base + (uint64_t)slot * h->per_rank_size + offset);
}

int moe_route_topk(const sym_heap *h, const float *logits, int32_t *idx, float *w,
                   symmoe_stream_t stream) {
  if (!heap_ok(h) || !aligned4(logits) || !aligned4(idx) || !aligned4(w)) return SYM_EINVAL;
  return from_cuda(launch_route_topk(*h, logits, idx, w, (cudaStream_t)stream));
}

int moe_router_logits(const sym_heap *h, const uint16_t *x, const uint16_t *w_router, float *logits,
                      symmoe_stream_t stream) {
  if (!heap_ok(h) || !aligned16(x) || !aligned16(w_router) || !aligned4(logits)) return SYM_EINVAL;
  const int sms = num_sms_of_current_device();
  if (sms <= 0) return SYM_ECUDA;
  return from_cuda(launch_router(*h, x, w_router, logits, sms, (cudaStream_t)stream));
}

int moe_router_splits(const sym_heap *h, int *splits) {
  if (!heap_ok(h) || !splits) return SYM_EINVAL;
  const int sms = num_sms_of_current_device();
  if (sms <= 0) return SYM_ECUDA;
  int grid, kb;
  return from_cuda(router_plan(*h, sms, &grid, splits, &kb));
}

int sym_gemm_a2a(const sym_heap *h, const uint16_t *x, const uint16_t *w, int mode, symmoe_stream_t stream) {
  if (!heap_ok(h) || !aligned16(x) || !aligned16(w) || (mode & ~SYM_LA_FUSED) ||
      h->s.tokens_per_slot % h->s.world != 0)
    return SYM_EINVAL;
  const int sms = num_sms_of_current_device();
  if (sms <= 0) return SYM_ECUDA;
  return from_cuda(launch_gemm_a2a(*h, x, w, mode & SYM_LA_FUSED, sms, (cudaStream_t)stream));
}

int sym_a2a_gemm(const sym_heap *h, const uint16_t *z, const uint16_t *w, int mode, symmoe_stream_t stream) {
  if (!heap_ok(h) || !aligned16(z) || !aligned16(w) || (mode & ~(SYM_LA_FUSED | SYM_LA_COPY_ENGINES)) ||
      mode == SYM_LA_COPY_ENGINES || h->s.hidden % (64 * h->s.world) != 0)
    return SYM_EINVAL;
  const bool engines = (mode & SYM_LA_COPY_ENGINES) != 0;
  if (engines && (uint32_t)a2a_gemm_counters(*h) > h->num_ready) return SYM_ENOSPACE;
  const int sms = num_sms_of_current_device();
  if (sms <= 0) return SYM_ECUDA;
  return from_cuda(launch_a2a_gemm(*h, z, w, engines ? 2 : (mode & SYM_LA_FUSED), sms, (cudaStream_t)stream));
}

int moe_dispatch(sym_heap *h, const uint16_t *x, const int32_t *idx, const float *w,
                 symmoe_stream_t stream) {
  return moe_dispatch_ex(h, x, idx, w, 0, stream);
}

// The deduplicated dispatch keeps its scratch in the h windows: per slot the
// row sources [cap], and in slot 0 also the chunk counts [W][N/32] and the
// pair ranks [N][k] (int32).
static bool dedup_fits(const sym_heap *h) {
  const uint64_t W = h->s.world, N = W * h->s.tokens_per_slot, k = h->s.topk;
  const uint64_t need = 4 * (h->cap + W * ((N + 31) / 32) + N * k);
  return W <= 32 && need <= h->cap * (uint64_t)h->s.inter * 2;
}

int moe_dispatch_ex(sym_heap *h, const uint16_t *x, const int32_t *idx, const float *w, int flags,
                    symmoe_stream_t stream) {
  if (!heap_ok(h) || !aligned16(x) || !aligned4(idx) || !aligned4(w) ||
      (flags & ~(SYM_DISPATCH_DEDUP | SYM_DISPATCH_FP8)) || flags == (SYM_DISPATCH_DEDUP | SYM_DISPATCH_FP8))
    return SYM_EINVAL;
  const int mode = (flags & SYM_DISPATCH_FP8) ? 2 : (flags & SYM_DISPATCH_DEDUP) ? 1 : 0;
  if (mode == 1 && !dedup_fits(h)) return SYM_EINVAL;
  h->epoch += 1;
  return from_cuda(launch_dispatch(*h, x, idx, w, mode, (cudaStream_t)stream));
}

int moe_expert_ffn_ex(const sym_heap *h, const uint16_t *w_gate, const uint16_t *w_up,
                      const uint16_t *w_down, int flags, symmoe_stream_t stream) {
  if (!heap_ok(h) || !aligned16(w_gate) || !aligned16(w_up) || !aligned16(w_down) ||
      (flags & ~SYM_FFN_WEIGHTED_ROWS))
    return SYM_EINVAL;
  const int sms = num_sms_of_current_device();
  if (sms <= 0) return SYM_ECUDA;
  return from_cuda(launch_expert_ffn(*h, w_gate, w_up, w_down, sms, 1, (flags & SYM_FFN_WEIGHTED_ROWS) ? 1 : 0,
                                     (cudaStream_t)stream));
}

int moe_expert_ffn(const sym_heap *h, const uint16_t *w_gate, const uint16_t *w_up,
                   const uint16_t *w_down, symmoe_stream_t stream) {
  return moe_expert_ffn_ex(h, w_gate, w_up, w_down, 0, stream);
}

int moe_combine_ex(const sym_heap *h, const uint16_t *expert_out, const int32_t *idx,
                   const float *w, uint16_t *out, int flags, symmoe_stream_t stream) {
  const bool unit = (flags & SYM_COMBINE_UNWEIGHTED) != 0;
  if (!heap_ok(h) || !aligned4(idx) || (!unit && !aligned4(w)) || !aligned16(out) ||
      (flags & ~SYM_COMBINE_UNWEIGHTED))
    return SYM_EINVAL;
  const uint16_t *view = reinterpret_cast<const uint16_t *>(h->base + h->off_y);
  const uint16_t *stage = nullptr;
  if (expert_out && expert_out != view) {
    if (!aligned16(expert_out)) return SYM_EINVAL;
    stage = expert_out;
    g_fallback_copies.fetch_add(1);
  }
  const int sms = num_sms_of_current_device();
  if (sms <= 0) return SYM_ECUDA;
  return from_cuda(launch_combine(*h, stage, idx, w, out, unit ? 1 : 0, sms, (cudaStream_t)stream));
}

int moe_combine(const sym_heap *h, const uint16_t *expert_out, const int32_t *idx,
                const float *w, uint16_t *out, symmoe_stream_t stream) {
  return moe_combine_ex(h, expert_out, idx, w, out, 0, stream);
}

uint64_t moe_combine_fallback_copies(void) { return g_fallback_copies.load(); }

int moe_pipeline(sym_heap *h, const float *logits, const uint16_t *x, const uint16_t *w_gate,
                 const uint16_t *w_up, const uint16_t *w_down, int32_t *idx, float *w,
                 uint16_t *out, int mode, symmoe_stream_t stream) {
  if (!heap_ok(h) || !aligned4(logits) || !aligned16(x) || !aligned16(w_gate) ||
      !aligned16(w_up) || !aligned16(w_down) || !aligned4(idx) || !aligned4(w) ||
      !aligned16(out) || (mode & ~(SYM_PIPE_FUSED | SYM_PIPE_WEIGHTS_IN_FFN | SYM_PIPE_DEDUP | SYM_PIPE_FP8)))
    return SYM_EINVAL;
  const int dmode = (mode & SYM_PIPE_FP8) ? 2 : (mode & SYM_PIPE_DEDUP) ? 1 : 0;
  if (dmode && ((mode & SYM_PIPE_FUSED) || ((mode & SYM_PIPE_DEDUP) && (mode & SYM_PIPE_FP8)) ||
                (dmode == 1 && !dedup_fits(h))))
    return SYM_EINVAL;
  const cudaStream_t st = (cudaStream_t)stream;
  const int sms = num_sms_of_current_device();
  if (sms <= 0) return SYM_ECUDA;
  const int weighted = (mode & SYM_PIPE_WEIGHTS_IN_FFN) ? 1 : 0;
  h->epoch += 1;
  if (mode & SYM_PIPE_FUSED)
    return from_cuda(launch_fused(*h, logits, x, w_gate, w_up, w_down, idx, w, out, weighted, sms, st));
  cudaError_t e = launch_route_topk(*h, logits, idx, w, st);
  if (e == cudaSuccess) e = launch_dispatch(*h, x, idx, w, dmode, st);
  if (e == cudaSuccess) e = launch_expert_ffn(*h, w_gate, w_up, w_down, sms, 1, weighted, st);
  if (e == cudaSuccess) e = launch_combine(*h, nullptr, idx, w, out, weighted, sms, st);
  return from_cuda(e);
}

int sym_heap_status(const sym_heap *h, int32_t *status, int clear, symmoe_stream_t stream) {
  if (!h || !status || h->base == 0) return SYM_EINVAL;
  const cudaStream_t st = (cudaStream_t)stream;
  int32_t *dev = reinterpret_cast<int32_t *>(h->base + h->off_status);
  if (cudaStreamSynchronize(st) != cudaSuccess) return SYM_ECUDA;
  if (cudaMemcpy(status, dev, sizeof(int32_t), cudaMemcpyDeviceToHost) != cudaSuccess)
    return SYM_ECUDA;
  if (clear && cudaMemset(dev, 0, sizeof(int32_t)) != cudaSuccess) return SYM_ECUDA;
  return SYM_OK;
}

// ---------------------------------------------------------------------------
// training through an MoE block
// ---------------------------------------------------------------------------
// rows of a tensor or a window: extents in range, rows that do not overlap
static bool rows_ok(const sym_rows *r, uint64_t align) {
  if (!r || r->slots < 1 || r->slots > 1024 || r->rows < 0 || r->cols < 1 || r->cols > 65536) return false;
  if (r->rows * r->slots >= (int64_t(1) << 30)) return false;
  if (r->rows > 0 && (r->ptr == 0 || r->ptr % align != 0)) return false;
  if (r->rows > 1 && r->ld < r->cols) return false;
  if (r->slots > 1 && r->rows > 0 && r->slot_stride < (r->rows - 1) * r->ld + r->cols) return false;
  return true;
}
// the tensor copies' rule: 16-byte aligned rows
static bool rows_tma_ok(const sym_rows *r) {
  return rows_ok(r, 16) && r->ld % 8 == 0 && r->ld >= r->cols && (r->slots == 1 || r->slot_stride % 8 == 0);
}
static bool same_rows(const sym_rows *a, const sym_rows *b) { return a->slots == b->slots && a->rows == b->rows; }
static bool groups_ok(const sym_groups *g, const sym_rows *r) {
  return g && aligned4(g->cnt) && aligned4(g->off) && g->groups >= 1 && g->groups <= 1024 && g->slots == r->slots &&
         g->groups % g->slots == 0 && (reinterpret_cast<uintptr_t>(g->status) & 3u) == 0 &&
         (g->slots == 1 || (g->cnt_slot_stride >= g->groups / g->slots && g->off_slot_stride >= g->groups / g->slots));
}
static sym_groups with_timeout(const sym_groups *g) {
  sym_groups c = *g;
  if (c.wait_timeout_us == 0) c.wait_timeout_us = kDefaultTimeoutUs;
  return c;
}

int moe_grouped_matmul(const sym_groups *g, int dtype, const sym_rows *x, const void *w, int64_t w_group_stride,
                       int64_t w_ld, int flags, const sym_rows *out, symmoe_stream_t stream) {
  if ((dtype != SYM_BF16 && dtype != SYM_FP16) || (flags & ~SYM_GM_TRANS_W) || !rows_tma_ok(x) || !rows_ok(out, 2) ||
      !same_rows(x, out) || !groups_ok(g, x) || !aligned16(w))
    return SYM_EINVAL;
  const int trans = flags & SYM_GM_TRANS_W;
  const int64_t w_rows = trans ? x->cols : out->cols, w_cols = trans ? out->cols : x->cols;
  if (w_ld % 8 != 0 || w_ld < w_cols ||
      (g->groups > 1 && (w_group_stride % 8 != 0 || w_group_stride < (w_rows - 1) * w_ld + w_cols)))
    return SYM_EINVAL;
  if (x->rows == 0) return SYM_OK;
  const int sms = num_sms_of_current_device();
  if (sms <= 0) return SYM_ECUDA;
  const auto launch = few_rows_product(*g, *x, trans)                ? launch_few_rows
                      : thin_product(*g, *x, *out, trans, sms) ? launch_thin_product
                                                               : launch_grouped_matmul;
  return from_cuda(launch(with_timeout(g), dtype == SYM_FP16, *x, w, w_group_stride, w_ld, trans, *out, sms,
                          (cudaStream_t)stream));
}

int moe_grouped_wgrad(const sym_groups *g, int dtype, const sym_rows *dy, const sym_rows *x, void *dw,
                      int64_t dw_group_stride, int64_t dw_ld, int out_dtype, int flags, symmoe_stream_t stream) {
  if ((dtype != SYM_BF16 && dtype != SYM_FP16) || (out_dtype != dtype && out_dtype != SYM_FP32) ||
      (flags & ~SYM_GM_ACCUMULATE) || !rows_tma_ok(dy) || !rows_tma_ok(x) || !same_rows(dy, x) || !groups_ok(g, x) ||
      !dw || reinterpret_cast<uintptr_t>(dw) % (out_dtype == SYM_FP32 ? 4 : 2) != 0 || dw_ld < x->cols ||
      (g->groups > 1 && dw_group_stride < (dy->cols - 1) * dw_ld + x->cols))
    return SYM_EINVAL;
  const int sms = num_sms_of_current_device();
  if (sms <= 0) return SYM_ECUDA;
  return from_cuda(launch_grouped_wgrad(with_timeout(g), dtype == SYM_FP16, *dy, *x, dw, dw_group_stride, dw_ld,
                                        out_dtype, flags & SYM_GM_ACCUMULATE, sms, (cudaStream_t)stream));
}

static bool dtype_ok(int dtype) { return dtype == SYM_BF16 || dtype == SYM_FP16 || dtype == SYM_FP32; }
static uint64_t size_of(int dtype) { return dtype == SYM_FP32 ? 4 : 2; }
static bool like_ok(const sym_rows *r, const sym_rows *first, int dtype) {
  return rows_ok(r, size_of(dtype)) && same_rows(r, first) && r->cols == first->cols;
}
static bool opt4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
static bool opt16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int moe_swiglu_rows(int dtype, const sym_rows *g, const sym_rows *u, const float *row_w, int64_t row_w_slot_stride,
                    const int32_t *total, int64_t total_slot_stride, const sym_rows *h, symmoe_stream_t stream) {
  if (!dtype_ok(dtype) || !rows_ok(g, size_of(dtype)) || !like_ok(u, g, dtype) || !like_ok(h, g, dtype) ||
      !opt4(row_w) || !opt4(total))
    return SYM_EINVAL;
  if (g->rows == 0) return SYM_OK;
  const int sms = num_sms_of_current_device();
  if (sms <= 0) return SYM_ECUDA;
  return from_cuda(launch_swiglu_rows(dtype, *g, *u, *h, row_w, row_w_slot_stride, total, total_slot_stride, sms,
                                      (cudaStream_t)stream));
}

int moe_swiglu_rows_bwd(int dtype, const sym_rows *g, const sym_rows *u, const sym_rows *dh, const float *row_w,
                        int64_t row_w_slot_stride, const int32_t *total, int64_t total_slot_stride,
                        const sym_rows *dg, const sym_rows *du, float *d_row_w, int64_t d_row_w_slot_stride,
                        symmoe_stream_t stream) {
  if (!dtype_ok(dtype) || !rows_ok(g, size_of(dtype)) || !like_ok(u, g, dtype) || !like_ok(dh, g, dtype) ||
      !like_ok(dg, g, dtype) || !like_ok(du, g, dtype) || !opt4(row_w) || !opt4(total) || !opt4(d_row_w))
    return SYM_EINVAL;
  if (g->rows == 0) return SYM_OK;
  const int sms = num_sms_of_current_device();
  if (sms <= 0) return SYM_ECUDA;
  return from_cuda(launch_swiglu_rows_bwd(dtype, *g, *u, *dh, *dg, *du, row_w, row_w_slot_stride, d_row_w,
                                          d_row_w_slot_stride, total, total_slot_stride, sms, (cudaStream_t)stream));
}

int moe_dropout(int dtype, const sym_rows *x, const sym_rows *residual, const sym_rows *y, double p, uint64_t seed,
                uint64_t offset, symmoe_stream_t stream) {
  if (!dtype_ok(dtype) || !rows_ok(x, size_of(dtype)) || !like_ok(y, x, dtype) ||
      (residual && !like_ok(residual, x, dtype)) || !(p >= 0.0 && p < 1.0))
    return SYM_EINVAL;
  if (x->rows == 0) return SYM_OK;
  const int sms = num_sms_of_current_device();
  if (sms <= 0) return SYM_ECUDA;
  return from_cuda(launch_dropout(dtype, *x, residual, *y, seed, offset, p, sms, (cudaStream_t)stream));
}

// a tensor of the call: aligned to its type, rows that do not overlap
static bool tensor_ok(const void *p, int64_t ld, int64_t rows, int cols, int dtype) {
  return reinterpret_cast<uintptr_t>(p) % size_of(dtype) == 0 &&
         (!p || rows <= 1 || (ld >= cols && ld < (int64_t(1) << 31)));
}
static bool block_ok(const sym_block_norm *a) {
  if (!a || !dtype_ok(a->dtype) || a->rows < 0 || a->rows >= (int64_t(1) << 30) || a->cols < 1 || a->cols > 65536)
    return false;
  if ((a->flags & ~SYM_NORM_NO_POST) || a->gate_act < SYM_GATE_NONE || a->gate_act > SYM_GATE_TANH) return false;
  if (!(a->p >= 0.0 && a->p < 1.0) || !(a->eps >= 0.f)) return false;
  if ((a->flags & SYM_NORM_NO_POST) && (a->w_post || a->rstd_post)) return false;
  // (an empty tensor may have no address)
  if (a->rows > 0 && !a->o && (a->w_post || a->gate || a->rstd_post)) return false;
  if (a->gate && (a->gate_rows < 1 || a->gate_rows >= (int64_t(1) << 31) ||
                  (a->rows > 0 && (a->gate_rows > a->rows || a->rows % a->gate_rows != 0))))
    return false;
  return tensor_ok(a->o, a->ld_o, a->rows, a->cols, a->dtype) && tensor_ok(a->y, a->ld_y, a->rows, a->cols, a->dtype) &&
         tensor_ok(a->gate, a->ld_gate, a->gate_rows, a->cols, a->dtype) &&
         tensor_ok(a->w_post, 0, 1, a->cols, a->dtype) && tensor_ok(a->w_pre, 0, 1, a->cols, a->dtype) &&
         opt4(a->rstd_post) && opt4(a->rstd_pre);
}

int moe_block_norm(const sym_block_norm *a, symmoe_stream_t stream) {
  if (!block_ok(a) || !tensor_ok(a->x, a->ld_x, a->rows, a->cols, a->dtype) ||
      !tensor_ok(a->h, a->ld_h, a->rows, a->cols, a->dtype))
    return SYM_EINVAL;
  if (a->rows == 0) return SYM_OK;
  if (!a->x || (a->o && !a->y) || (!a->o && a->y) || (!a->o && !a->h && !a->rstd_pre)) return SYM_EINVAL;
  const int sms = num_sms_of_current_device();
  if (sms <= 0) return SYM_ECUDA;
  return from_cuda(launch_block_norm(*a, sms, (cudaStream_t)stream));
}

int moe_block_norm_workspace(int64_t rows, int32_t cols, int64_t gate_rows, uint64_t *bytes) {
  if (!bytes || rows < 0 || rows >= (int64_t(1) << 30) || cols < 1 || cols > 65536 || gate_rows < 0 ||
      (gate_rows > 0 && rows > 0 && (gate_rows > rows || rows % gate_rows != 0)))
    return SYM_EINVAL;
  const int sms = num_sms_of_current_device();
  if (sms <= 0) return SYM_ECUDA;
  *bytes = rows == 0 ? 0 : block_norm_workspace(rows, cols, gate_rows, sms);
  return SYM_OK;
}

int moe_block_norm_bwd(const sym_block_norm *a, const sym_block_norm_grad *g, symmoe_stream_t stream) {
  if (!block_ok(a) || !g) return SYM_EINVAL;
  const int64_t R = a->rows;
  const int C = a->cols, t = a->dtype;
  if (!tensor_ok(g->dy, g->ld_dy, R, C, t) || !tensor_ok(g->dh, g->ld_dh, R, C, t) ||
      !tensor_ok(g->dx, g->ld_dx, R, C, t) || !tensor_ok(g->d_o, g->ld_do, R, C, t) ||
      !tensor_ok(g->dw_pre, 0, 1, C, t) || !tensor_ok(g->dw_post, 0, 1, C, t) ||
      !tensor_ok(g->dgate, g->ld_dgate, a->gate_rows, C, t) || (reinterpret_cast<uintptr_t>(g->work) & 15u))
    return SYM_EINVAL;
  if ((!a->gate && g->dgate) || ((a->flags & SYM_NORM_NO_POST) && g->dw_post)) return SYM_EINVAL;
  if (R == 0) {  // sums over no rows
    const cudaStream_t st = (cudaStream_t)stream;
    const size_t row = C * size_of(t);
    cudaError_t e = cudaSuccess;
    if (g->dw_pre) e = cudaMemsetAsync(g->dw_pre, 0, row, st);
    if (e == cudaSuccess && g->dw_post) e = cudaMemsetAsync(g->dw_post, 0, row, st);
    if (e == cudaSuccess && g->dgate) {
      const size_t pitch = a->gate_rows > 1 ? g->ld_dgate * size_of(t) : row;
      e = cudaMemset2DAsync(g->dgate, pitch, 0, row, (size_t)a->gate_rows, st);
    }
    return from_cuda(e);
  }
  if ((!a->o && (g->d_o || g->dw_post)) || (!g->dy && !g->dh) || (g->dh && (!a->y || !a->rstd_pre)) || (!g->dh && g->dw_pre) ||
      (a->o && !(a->flags & SYM_NORM_NO_POST) && !a->rstd_post))
    return SYM_EINVAL;
  const int sms = num_sms_of_current_device();
  if (sms <= 0) return SYM_ECUDA;
  if (!g->work || g->work_bytes < block_norm_workspace(R, C, g->dgate ? a->gate_rows : 0, sms)) return SYM_ENOSPACE;
  return from_cuda(launch_block_norm_bwd(*a, *g, sms, (cudaStream_t)stream));
}

// ---------------------------------------------------------------------------
// layer norm, updates of the experts' matrices, a few tokens
// ---------------------------------------------------------------------------
static bool norm_shape_ok(int64_t rows, int cols) { return rows >= 0 && rows < (int64_t(1) << 30) && cols >= 1 && cols <= 65536; }

int moe_layer_norm(const sym_layer_norm *a, symmoe_stream_t stream) {
  if (!a || !dtype_ok(a->dtype) || !norm_shape_ok(a->rows, a->cols) || !(a->eps >= 0.f)) return SYM_EINVAL;
  const int64_t R = a->rows;
  const int C = a->cols, t = a->dtype;
  if (!tensor_ok(a->x, a->ld_x, R, C, t) || !tensor_ok(a->add, a->ld_add, R, C, t) || !tensor_ok(a->sum, a->ld_sum, R, C, t) ||
      !tensor_ok(a->h, a->ld_h, R, C, t) || !tensor_ok(a->w, 0, 1, C, t) || !tensor_ok(a->b, 0, 1, C, t) || !opt4(a->mean) ||
      !opt4(a->rstd))
    return SYM_EINVAL;
  if (R == 0) return SYM_OK;
  if (!a->x || (!a->h && !a->sum && !a->mean && !a->rstd) || (a->h && a->h == a->sum)) return SYM_EINVAL;
  const int sms = num_sms_of_current_device();
  if (sms <= 0) return SYM_ECUDA;
  return from_cuda(launch_layer_norm(*a, sms, (cudaStream_t)stream));
}

int moe_layer_norm_workspace(int64_t rows, int32_t cols, uint64_t *bytes) {
  if (!bytes || !norm_shape_ok(rows, cols)) return SYM_EINVAL;
  const int sms = num_sms_of_current_device();
  if (sms <= 0) return SYM_ECUDA;
  *bytes = rows == 0 ? 0 : layer_norm_workspace(rows, cols, sms);
  return SYM_OK;
}

int moe_layer_norm_bwd(const sym_layer_norm_grad *a, symmoe_stream_t stream) {
  if (!a || !dtype_ok(a->dtype) || !norm_shape_ok(a->rows, a->cols)) return SYM_EINVAL;
  const int64_t R = a->rows;
  const int C = a->cols, t = a->dtype;
  if (!tensor_ok(a->dh, a->ld_dh, R, C, t) || !tensor_ok(a->s, a->ld_s, R, C, t) || !tensor_ok(a->dsum, a->ld_dsum, R, C, t) ||
      !tensor_ok(a->dx, a->ld_dx, R, C, t) || !tensor_ok(a->w, 0, 1, C, t) || !tensor_ok(a->dw, 0, 1, C, t) ||
      !tensor_ok(a->db, 0, 1, C, t) || !opt4(a->mean) || !opt4(a->rstd) || !opt16(a->work))
    return SYM_EINVAL;
  if (!a->dx && !a->dw && !a->db) return SYM_EINVAL;
  if (R == 0) {  // sums over no rows
    const cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e = cudaSuccess;
    if (a->dw) e = cudaMemsetAsync(a->dw, 0, C * size_of(t), st);
    if (e == cudaSuccess && a->db) e = cudaMemsetAsync(a->db, 0, C * size_of(t), st);
    return from_cuda(e);
  }
  if (!a->dh || !a->s || !a->mean || !a->rstd) return SYM_EINVAL;
  const int sms = num_sms_of_current_device();
  if (sms <= 0) return SYM_ECUDA;
  if ((a->dw || a->db) && (!a->work || a->work_bytes < layer_norm_workspace(R, C, sms))) return SYM_ENOSPACE;
  return from_cuda(launch_layer_norm_bwd(*a, sms, (cudaStream_t)stream));
}

static bool orth_shape_ok(int count, int rows, int cols) {
  return count >= 0 && count <= 65535 && rows >= 1 && rows <= 65536 && cols >= 1 && cols <= 65536;
}
// matrices of a batch: aligned to their type, rows and matrices that do not overlap
static bool matrices_ok(const void *p, int count, int rows, int cols, int64_t stride, int64_t ld, int dtype) {
  return p && reinterpret_cast<uintptr_t>(p) % size_of(dtype) == 0 && (rows == 1 || ld >= cols) &&
         (count == 1 || stride >= (rows - 1) * (rows == 1 ? 0 : ld) + cols);
}

int moe_orthogonalize_workspace(int32_t count, int32_t rows, int32_t cols, uint64_t *work_bytes, uint64_t *least_bytes) {
  if (!orth_shape_ok(count, rows, cols) || (!work_bytes && !least_bytes)) return SYM_EINVAL;
  const int sms = num_sms_of_current_device();
  if (sms <= 0) return SYM_ECUDA;
  size_t least = 0, best = 0;
  orthogonalize_workspace(count, rows, cols, sms, &least, &best);
  if (work_bytes) *work_bytes = best;
  if (least_bytes) *least_bytes = least;
  return SYM_OK;
}

int moe_orthogonalize(const sym_orthogonalize *a, symmoe_stream_t stream) {
  if (!a || !orth_shape_ok(a->count, a->rows, a->cols) || a->steps < 0 || a->steps > 64 || !dtype_ok(a->g_dtype) ||
      (a->out_dtype != SYM_BF16 && a->out_dtype != SYM_FP16) || !(a->eps >= 0.f) || (reinterpret_cast<uintptr_t>(a->work) & 255u) || !opt4(a->status))
    return SYM_EINVAL;
  if (a->count == 0) return SYM_OK;
  if (!matrices_ok(a->g, a->count, a->rows, a->cols, a->g_stride, a->ld_g, a->g_dtype) ||
      !matrices_ok(a->out, a->count, a->rows, a->cols, a->out_stride, a->ld_out, a->out_dtype))
    return SYM_EINVAL;
  const int sms = num_sms_of_current_device();
  if (sms <= 0) return SYM_ECUDA;
  size_t least = 0, best = 0;
  orthogonalize_workspace(a->count, a->rows, a->cols, sms, &least, &best);
  if (!a->work || a->work_bytes < least) return SYM_ENOSPACE;
  return from_cuda(launch_orthogonalize(*a, sms, (cudaStream_t)stream));
}

static bool few_shape_ok(int tokens, int inter, int topk) {
  return tokens >= 0 && tokens <= 32 && inter >= 8 && inter <= 65536 && inter % 8 == 0 && topk >= 1 && topk <= 32;
}
// an expert's matrices: 16-byte aligned rows, none over another
static bool expert_ok(const void *p, int experts, int rows, int cols, int64_t group, int64_t ld) {
  return aligned16(p) && ld % 8 == 0 && ld >= cols && (experts == 1 || (group % 8 == 0 && group >= (rows - 1) * ld + cols));
}

int moe_few_tokens_workspace(int32_t tokens, int32_t inter, int32_t topk, uint64_t *bytes) {
  if (!bytes || !few_shape_ok(tokens, inter, topk)) return SYM_EINVAL;
  *bytes = few_tokens_workspace(tokens, inter, topk);
  return SYM_OK;
}

int moe_few_tokens(const sym_few_tokens *a, symmoe_stream_t stream) {
  if (!a || !few_shape_ok(a->tokens, a->inter, a->topk) || a->hidden < 8 || a->hidden > 65536 || a->hidden % 8 != 0 ||
      a->num_experts < 1 || a->num_experts > 1024 || a->topk > a->num_experts || (a->dtype != SYM_BF16 && a->dtype != SYM_FP16))
    return SYM_EINVAL;
  const int T = a->tokens, H = a->hidden, I = a->inter, E = a->num_experts;
  if (!expert_ok(a->w_gate, E, I, H, a->gate_group, a->gate_ld) || !expert_ok(a->w_up, E, I, H, a->up_group, a->up_ld) ||
      !expert_ok(a->w_down, E, H, I, a->down_group, a->down_ld) || (a->w_router && !expert_ok(a->w_router, 1, E, H, 0, a->router_ld)) ||
      !opt16(a->work))
    return SYM_EINVAL;
  if (T == 0) return SYM_OK;
  if (!aligned16(a->x) || (T > 1 && (a->ld_x % 8 != 0 || a->ld_x < H)) || !a->out || (reinterpret_cast<uintptr_t>(a->out) & 1u) ||
      (T > 1 && a->ld_out < H) || !aligned4(a->logits) || !aligned4(a->idx) || !aligned4(a->w))
    return SYM_EINVAL;
  const int sms = num_sms_of_current_device();
  if (sms <= 0) return SYM_ECUDA;
  if (!a->work || a->work_bytes < few_tokens_workspace(T, I, a->topk)) return SYM_ENOSPACE;
  return from_cuda(launch_few_tokens(*a, sms, (cudaStream_t)stream));
}

const char *sym_strerror(int code) {
  switch (code) {
    case SYM_OK: return "success";
    case SYM_EINVAL: return "invalid shape, pointer, alignment or argument";
    case SYM_ENOSPACE: return "heap (or a window of it) too small for the call";
    case SYM_ECUDA: return "CUDA runtime call or kernel launch failed";
    case SYM_ETIMEOUT: return "a bounded device wait expired";
    case SYM_EOVERFLOW: return "a row or expert index out of range";
    case SYM_ENOTSUP: return "not supported on this device";
    default: return "unknown symmoe status code";
  }
}

}  // extern "C"
