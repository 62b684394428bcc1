// C ABI of the paged KV cache (include/dg.h, dg_paged_*): argument checks on
// the host, launch shapes, and the choice of the attention kernel.  Included
// by engine.cu, whose tensor-map helpers it uses and whose ragged batches make
// the same launches.
#pragma once

#include <atomic>
#include <initializer_list>

#include "paged.cuh"
#include "paged_attention.cuh"
#include "paged_canvas.cuh"

namespace {

// the plan's CTAs: one per SM of a B200 (another number costs time, not the result)
constexpr int kPlanCtas = 148;

// log2 of a supported page size, -1 for any other
int page_shift_of(int32_t page_size) {
  switch (page_size) {
    case 16: return 4;
    case 32: return 5;
    case 64: return 6;
    case 128: return 7;
    default: return -1;
  }
}

// heads the paged kernels serve: the shapes of dg_config
dg_status check_heads(int Hq, int Hkv, int D) {
  if (Hq <= 0 || Hkv <= 0 || D <= 0) return DG_ERR_INVALID_ARG;
  if ((D != 64 && D != 128 && D != 176) || Hq % Hkv || ATC_BQ % (Hq / Hkv) || Hq > 1024) return DG_ERR_UNSUPPORTED;
  return DG_OK;
}

// a call's operand in device memory
struct Operand {
  const void* at;
  int64_t bytes;
  bool written;
};

// Whether some written operand shares memory with another one: other CTAs may
// still read what it overwrites.
bool operands_clash(std::initializer_list<Operand> list) {
  for (const Operand* a = list.begin(); a != list.end(); ++a)
    for (const Operand* b = a + 1; b != list.end(); ++b) {
      const uintptr_t x = reinterpret_cast<uintptr_t>(a->at), y = reinterpret_cast<uintptr_t>(b->at);
      if ((a->written || b->written) && a->bytes > 0 && b->bytes > 0 && x < y + b->bytes && y < x + a->bytes)
        return true;
    }
  return false;
}

// a launch's own status; an error that the caller left pending is neither
// reported nor cleared
template <typename P>
dg_status paged_launch(void (*kernel)(P), dim3 grid, int threads, size_t smem, void* stream, const P& p) {
  cudaLaunchConfig_t lc{};
  lc.gridDim = grid;
  lc.blockDim = dim3(threads);
  lc.dynamicSmemBytes = smem;
  lc.stream = static_cast<cudaStream_t>(stream);
  // it may start while the kernel before it still runs, and waits for its end itself
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = &attr;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, kernel, p) == cudaSuccess ? DG_OK : DG_ERR_CUDA;
}

template <bool SPLITS>
dg_status launch_append(const PagedAppendParams& p, int head_dim, void* stream) {
  const int groups = (p.Hq + 2 * p.Hkv + APPEND_HEADS - 1) / APPEND_HEADS;
  const int64_t grid = (static_cast<int64_t>(p.rows) * groups * (head_dim / 16) + APPEND_THREADS - 1) / APPEND_THREADS;
  if (grid > INT32_MAX) return DG_ERR_CAPACITY;
  auto* kern = head_dim == 64 ? paged_append_kernel<64, SPLITS>
               : head_dim == 128 ? paged_append_kernel<128, SPLITS> : paged_append_kernel<176, SPLITS>;
  return paged_launch(kern, dim3(static_cast<unsigned>(grid)), APPEND_THREADS, 0, stream, p);
}

// What the attention calls need of a device: its SM count, and the kernels'
// shared-memory limits raised once (under a lock; the first call on a device
// may come from any thread, and may be captured: neither is a stream
// operation).
struct PagedSetup {
  std::atomic<int> sms{0};
};
PagedSetup g_paged_setup[kMaxDevices];
std::mutex g_paged_setup_mutex;

static_assert(TokCfg<64>::SMEM <= kMaxSmemPerCta && TokCfg<128>::SMEM <= kMaxSmemPerCta &&
                  TokCfg<176>::SMEM <= kMaxSmemPerCta,
              "token attention shared memory");
static_assert(CvCfg<64>::SMEM <= kMaxSmemPerCta && CvCfg<128>::SMEM <= kMaxSmemPerCta &&
                  CvCfg<176>::SMEM <= kMaxSmemPerCta,
              "canvas attention shared memory");

template <typename K>
bool raise_smem(K* kernel, int bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess;
}

// SM count of the current device, 0 if it cannot be had
int paged_device_sms() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  PagedSetup& g = g_paged_setup[dev];
  int sms = g.sms.load(std::memory_order_acquire);
  if (sms) return sms;
  std::lock_guard<std::mutex> lock(g_paged_setup_mutex);
  sms = g.sms.load(std::memory_order_relaxed);
  if (sms) return sms;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
      !raise_smem(paged_token_kernel<64>, TokCfg<64>::SMEM) ||
      !raise_smem(paged_token_kernel<128>, TokCfg<128>::SMEM) ||
      !raise_smem(paged_token_kernel<176>, TokCfg<176>::SMEM) ||
      !raise_smem(paged_canvas_kernel<64>, CvCfg<64>::SMEM) ||
      !raise_smem(paged_canvas_kernel<128>, CvCfg<128>::SMEM) ||
      !raise_smem(paged_canvas_kernel<176>, CvCfg<176>::SMEM))
    return 0;
  g.sms.store(sms, std::memory_order_release);
  return sms;
}

// host checks of dg_paged_attention that need no workspace
dg_status check_attention(const dg_paged_attention_args* a) {
  if (!a || !a->q || !a->k_pages || !a->v_pages || !a->block_table || !a->kv_lens || !a->cu_rows || !a->out ||
      a->n_rows < 0 || a->batch <= 0 || a->n_pages <= 0 || a->table_width <= 0 || a->table_stride < a->table_width ||
      !(a->scale > 0.f) || !(a->scale < INFINITY) || !aligned16(a->q) || !aligned16(a->k_pages) ||
      !aligned16(a->v_pages) || !aligned16(a->out))
    return DG_ERR_INVALID_ARG;
  const dg_status hs = check_heads(a->n_q_heads, a->n_kv_heads, a->head_dim);
  if (hs != DG_OK) return hs;
  const int shift = page_shift_of(a->page_size);
  if (shift < 0) return DG_ERR_UNSUPPORTED;
  if (a->q_stride < static_cast<int64_t>(a->n_q_heads) * a->head_dim || a->q_stride % 8) return DG_ERR_INVALID_ARG;
  // TMA row coordinates and key positions are 32 bits
  if (static_cast<int64_t>(a->n_pages) * a->n_kv_heads > (INT32_MAX >> shift) ||
      a->table_width > (INT32_MAX >> shift))
    return DG_ERR_CAPACITY;
  return DG_OK;
}

// Tiles of 16 packed rows for requests whose rows fit one (they are bound by
// the stream of pages), of 256 on the tensor cores' accumulators above it.
bool few_rows(int64_t rows, int64_t max_rows, int G) {
  return (max_rows > 0 && max_rows < rows ? max_rows : rows) * G <= TOK_ROWS;
}

int64_t paged_workspace(bool few, int head_dim, int sms) {
  const int64_t rows = few ? TOK_ROWS : CV_ROWS;
  return 2 * sms * rows * (head_dim * 4 + 8) + sms * static_cast<int64_t>(sizeof(PagedCut));
}

// Queries [row][Hq][D] seen as (D, G, Hkv, row): a box of 64 columns x G heads
// x 1 kv head x 128 / G rows is the 128 packed rows of one GQA group.
bool make_map_rows(CUtensorMap* m, const dg_paged_attention_args* a) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t D = a->head_dim, G = a->n_q_heads / a->n_kv_heads;
  cuuint64_t dims[4] = {D, G, static_cast<cuuint64_t>(a->n_kv_heads), static_cast<cuuint64_t>(a->n_rows)};
  cuuint64_t strides[3] = {D * 2, G * D * 2, static_cast<cuuint64_t>(a->q_stride) * 2};
  cuuint32_t box[4] = {64, static_cast<cuuint32_t>(G), 1, static_cast<cuuint32_t>(CV_TILE / G)};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(a->q), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// the merge's CTAs: one per tile where the call has no more tiles than the device SMs, else one per SM
template <int ROWS, int D>
dg_status launch_merge(const PagedAttnParams& p, int tiles, int sms, void* stream) {
  using C = MergeCfg<ROWS>;
  const dim3 grid(p.cuts_by_tile ? tiles : sms, ROWS == TOK_ROWS ? 1 : D / 4 / C::COLS);
  return paged_launch(paged_merge_kernel<ROWS, D>, grid, C::THREADS, 0, stream, p);
}

template <int D>
dg_status launch_token(const PagedAttnParams& p, int tiles, int sms, void* stream) {
  const dg_status st = paged_launch(paged_token_kernel<D>, dim3(sms), TOK_THREADS, TokCfg<D>::SMEM, stream, p);
  return st != DG_OK ? st : launch_merge<TOK_ROWS, D>(p, tiles, sms, stream);
}

template <int D>
dg_status launch_canvas(const CanvasParams& p, int tiles, int sms, void* stream) {
  const dg_status st = paged_launch(paged_canvas_kernel<D>, dim3(sms), CV_THREADS, CvCfg<D>::SMEM, stream, p);
  return st != DG_OK ? st : launch_merge<CV_ROWS, D>(p.a, tiles, sms, stream);
}

// Attention with everything of p set but the workspace's parts and the lists:
// the kernel for tiles of 16 or of 256 rows, then the merge.
dg_status launch_attention(CanvasParams& cp, bool few, int head_dim, void* workspace, int sms, void* stream) {
  PagedAttnParams& p = cp.a;
  const int64_t tile_rows = few ? TOK_ROWS : CV_ROWS, slots = 2 * static_cast<int64_t>(sms) * tile_rows;
  p.g_shift = 0;
  while (p.Hkv << p.g_shift < p.Hq) ++p.g_shift;
  p.part = static_cast<float*>(workspace);
  p.part_ml = reinterpret_cast<float2*>(p.part + slots * head_dim);
  p.cuts = reinterpret_cast<PagedCut*>(p.part_ml + slots);
  // tiles: ceil(rows_b * G / ROWS) over the requests, per kv head
  const int64_t tiles64 = (static_cast<int64_t>(p.rows) * (p.Hq / p.Hkv) / tile_rows + p.batch) * p.Hkv;
  const int tiles = static_cast<int>(std::min<int64_t>(tiles64, sms));
  p.cuts_by_tile = tiles64 <= sms ? tiles : 0;
  switch (head_dim) {
    case 64: return few ? launch_token<64>(p, tiles, sms, stream) : launch_canvas<64>(cp, tiles, sms, stream);
    case 128: return few ? launch_token<128>(p, tiles, sms, stream) : launch_canvas<128>(cp, tiles, sms, stream);
    default: return few ? launch_token<176>(p, tiles, sms, stream) : launch_canvas<176>(cp, tiles, sms, stream);
  }
}

}  // namespace

extern "C" {

dg_status dg_paged_plan(const dg_paged_plan_args* a, void* cuda_stream) {
  if (!a || !a->cached_lens || !a->new_rows || !a->block_table || !a->free_pages || !a->free_state || !a->cu_rows ||
      !a->kv_lens || !a->free_state_out || a->batch <= 0 || a->table_width <= 0 ||
      a->table_stride < a->table_width || a->n_pages <= 0 || a->row_capacity < 0 ||
      (a->row_capacity > 0 && (!a->positions || !a->slots)))
    return DG_ERR_INVALID_ARG;
  const int shift = page_shift_of(a->page_size);
  if (shift < 0) return DG_ERR_UNSUPPORTED;
  if (a->n_pages > (INT32_MAX >> shift)) return DG_ERR_CAPACITY;  // a slot is 32 bits
  const int64_t B = a->batch, cap = a->row_capacity;
  if (operands_clash({{a->cached_lens, B * 4, false},
                      {a->new_rows, B * 4, false},
                      {a->free_state, 8, false},
                      {a->block_table, ((B - 1) * a->table_stride + a->table_width) * 4, true},
                      {a->free_pages, a->n_pages * int64_t(4), true},
                      {a->cu_rows, (B + 1) * 4, true},
                      {a->kv_lens, B * 4, true},
                      {a->positions, cap * 4, true},
                      {a->slots, cap * 4, true},
                      {a->free_state_out, 16, true}}))
    return DG_ERR_INVALID_ARG;
  PagedPlanParams p;
  p.cached = a->cached_lens;
  p.fresh = a->new_rows;
  p.table = a->block_table;
  p.table_stride = a->table_stride;
  p.ring = a->free_pages;
  p.state = a->free_state;
  p.cu_rows = a->cu_rows;
  p.kv_lens = a->kv_lens;
  p.positions = a->positions;
  p.slots = a->slots;
  p.state_out = a->free_state_out;
  p.batch = a->batch;
  p.width = a->table_width;
  p.n_pages = a->n_pages;
  p.page_shift = shift;
  p.row_cap = a->row_capacity;
  // one CTA per request up to a wave of them; strips of a request's rows where
  // there are few requests of many rows
  const int gx = std::min<int>(a->batch, kPlanCtas);
  const int64_t strips = cap / (B * 2 * PLAN_THREADS);
  const int gy = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(strips, kPlanCtas / gx)));
  return paged_launch(paged_plan_kernel, dim3(gx, gy), PLAN_THREADS, 0, cuda_stream, p);
}

dg_status dg_paged_append(const dg_paged_append_args* a, void* cuda_stream) {
  if (!a || !a->qkv || !a->positions || !a->slots || !a->rope || !a->k_pages || !a->v_pages || !a->q_out ||
      a->n_rows < 0 || a->n_positions <= 0 || a->n_pages <= 0 || !aligned16(a->qkv) || !aligned16(a->rope) ||
      !aligned16(a->k_pages) || !aligned16(a->v_pages) || !aligned16(a->q_out))
    return DG_ERR_INVALID_ARG;
  const dg_status hs = check_heads(a->n_q_heads, a->n_kv_heads, a->head_dim);
  if (hs != DG_OK) return hs;
  const int shift = page_shift_of(a->page_size);
  if (shift < 0) return DG_ERR_UNSUPPORTED;
  const int64_t rows = a->n_rows, width = (a->n_q_heads + int64_t(2) * a->n_kv_heads) * a->head_dim;
  if (a->qkv_stride < width || a->qkv_stride % 8) return DG_ERR_INVALID_ARG;
  if (a->n_pages > (INT32_MAX >> shift)) return DG_ERR_CAPACITY;
  if (rows == 0) return DG_OK;
  const int64_t pool = (static_cast<int64_t>(a->n_pages) << shift) * a->n_kv_heads * a->head_dim * 2;
  if (operands_clash({{a->qkv, ((rows - 1) * a->qkv_stride + width) * 2, false},
                      {a->positions, rows * 4, false},
                      {a->slots, rows * 4, false},
                      {a->rope, static_cast<int64_t>(a->n_positions) * a->head_dim * 4, false},
                      {a->k_pages, pool, true},
                      {a->v_pages, pool, true},
                      {a->q_out, rows * a->n_q_heads * a->head_dim * 2, true}}))
    return DG_ERR_INVALID_ARG;
  PagedAppendParams p{};
  p.qkv = static_cast<const uint16_t*>(a->qkv);
  p.qkv_stride = a->qkv_stride;
  p.positions = a->positions;
  p.slots = a->slots;
  p.rope = reinterpret_cast<const float4*>(a->rope);
  p.k = static_cast<uint16_t*>(a->k_pages);
  p.v = static_cast<uint16_t*>(a->v_pages);
  p.q = static_cast<uint16_t*>(a->q_out);
  p.n_slots = static_cast<int64_t>(a->n_pages) << shift;
  p.rows = a->n_rows;
  p.n_positions = a->n_positions;
  p.Hq = a->n_q_heads;
  p.Hkv = a->n_kv_heads;
  p.page_shift = shift;
  return launch_append<false>(p, a->head_dim, cuda_stream);
}

dg_status dg_paged_attention_workspace(const dg_paged_attention_args* a, int64_t* bytes) {
  const dg_status st = check_attention(a);
  if (st != DG_OK || !bytes) return bytes ? st : DG_ERR_INVALID_ARG;
  const int sms = paged_device_sms();
  if (!sms) return DG_ERR_CUDA;
  *bytes = paged_workspace(few_rows(a->n_rows, a->max_rows, a->n_q_heads / a->n_kv_heads), a->head_dim, sms);
  return DG_OK;
}

dg_status dg_paged_attention(const dg_paged_attention_args* a, void* cuda_stream) {
  const dg_status cs = check_attention(a);
  if (cs != DG_OK) return cs;
  if (a->n_rows == 0) return DG_OK;
  if (!a->workspace || !aligned16(a->workspace)) return DG_ERR_INVALID_ARG;
  const int sms = paged_device_sms();
  if (!sms) return DG_ERR_CUDA;
  const bool few = few_rows(a->n_rows, a->max_rows, a->n_q_heads / a->n_kv_heads);
  if (a->workspace_bytes < paged_workspace(few, a->head_dim, sms)) return DG_ERR_CAPACITY;
  const int shift = page_shift_of(a->page_size);
  const int64_t rows = a->n_rows, width = static_cast<int64_t>(a->n_q_heads) * a->head_dim;
  const int64_t pool = (static_cast<int64_t>(a->n_pages) << shift) * a->n_kv_heads * a->head_dim * 2;
  if (operands_clash({{a->q, ((rows - 1) * a->q_stride + width) * 2, false},
                      {a->k_pages, pool, false},
                      {a->v_pages, pool, false},
                      {a->block_table, ((a->batch - 1) * a->table_stride + a->table_width) * 4, false},
                      {a->kv_lens, a->batch * int64_t(4), false},
                      {a->cu_rows, (a->batch + int64_t(1)) * 4, false},
                      {a->out, rows * width * 2, true},
                      {a->lse, a->lse ? rows * a->n_q_heads * 4 : 0, true},
                      {a->workspace, paged_workspace(few, a->head_dim, sms), true}}))
    return DG_ERR_INVALID_ARG;
  CanvasParams cp;
  PagedAttnParams& p = cp.a;
  const uint64_t pool_rows = (static_cast<uint64_t>(a->n_pages) * a->n_kv_heads) << shift;
  const uint32_t box = std::min(a->page_size, PG_BK);
  if (!make_map(&p.k_map, a->k_pages, pool_rows, a->head_dim, box) ||
      !make_map(&p.v_map, a->v_pages, pool_rows, a->head_dim, box) || (!few && !make_map_rows(&cp.q_map, a)))
    return DG_ERR_CUDA;
  p.q = static_cast<const uint16_t*>(a->q);
  p.q_stride = a->q_stride;
  p.table = a->block_table;
  p.table_stride = a->table_stride;
  p.kv_lens = a->kv_lens;
  p.cu_rows = a->cu_rows;
  p.o = static_cast<uint16_t*>(a->out);
  p.lse = a->lse;
  p.rows = a->n_rows;
  p.batch = a->batch;
  p.Hq = a->n_q_heads;
  p.Hkv = a->n_kv_heads;
  p.n_pages = a->n_pages;
  p.page_shift = shift;
  p.width = a->table_width;
  p.causal = a->causal != 0;
  p.scale_log2 = static_cast<float>(1.4426950408889634 * static_cast<double>(a->scale));
  p.err = DevErr{nullptr, 1000000000ull};
  return launch_attention(cp, few, a->head_dim, a->workspace, sms, cuda_stream);
}

}  // extern "C"
