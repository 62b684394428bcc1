// Attention of packed rows over paged keys and values.  Row i of request b (n
// rows, kv keys) sees keys [0, kv), or with `causal` [0, kv - n + i + 1):
//   o = softmax(scale q K^T) V over them, lse = log sum exp of its scores.
// Keys of a page id outside the pool count as masked; a row that sees nothing
// gives zeros and lse = -inf.
//
// Work is counted in units: one 64-key block of one tile (packed rows of one
// request and kv head).  The units of a call form one line, in the order
// (request, row tile, kv head, key block), and the CTAs take stretches of equal
// length of it: every CTA has the same work whatever the requests' lengths, and
// the lengths are read on the device, so a captured launch serves any.  A tile
// that a stretch cuts leaves its raw rows and row statistics in a partial slot
// (two per CTA: the stretch's first tile and its last), and the merge kernel
// joins them in key order.
#pragma once

#include "paged.cuh"

namespace dg {

constexpr int PG_BK = 64;      // keys per unit

// A tile that a CTA's stretch begins and the next ones finish; rows = 0: none.
struct PagedCut {
  int rows;                    // live packed rows of the tile
  int t0, row0, h;             // the request's first row, the tile's first packed row, kv head
  int first, slot;             // CTA and partial slot of the first piece
  int last;                    // CTA of the last piece (the pieces between: slot 2 c of CTA c)
  int tiles;                   // tiles of the whole call
};

struct PagedAttnParams {
  CUtensorMap k_map;           // 2-D (D, n_pages * Hkv * page_size) over the pool; box (64, min(page_size, 64))
  CUtensorMap v_map;
  const uint16_t* q;           // [rows][Hq][D], row stride q_stride
  int64_t q_stride;
  const int32_t* table;
  int64_t table_stride;
  const int32_t* kv_lens;
  const int32_t* cu_rows;
  uint16_t* o;                 // [rows][Hq][D]
  float* lse;                  // [rows][Hq] or null
  float* part;                 // [CTA][2][tile rows][D] raw rows of cut tiles
  float2* part_ml;             // [CTA][2][tile rows] their (max in log2 units, sum)
  PagedCut* cuts;              // [CTA], or with cuts_by_tile [tile]
  int rows, batch, Hq, Hkv, n_pages, page_shift, width, causal;
  int g_shift;                 // log2 of the group size Hq / Hkv, a divisor of 128
  int cuts_by_tile;            // entries of `cuts` by tile where the call has at most as many tiles as CTAs, else 0
  float scale_log2;            // log2(e) * scale
  DevErr err;
};

struct PagedRequest {
  int t0, n, kv, tiles;        // first row, rows, keys (of those the table holds), row tiles
  int before;                  // keys before the first row's own; less than -1 where the first rows see none
};

template <int ROWS>
__host__ __device__ __forceinline__ PagedRequest paged_request(const PagedAttnParams& p, int b) {
  PagedRequest r;
  r.t0 = min(max(p.cu_rows[b], 0), p.rows);
  r.n = min(max(p.cu_rows[b + 1], r.t0), p.rows) - r.t0;   // within the call whatever the entry, and no overflow
  const int len = max(p.kv_lens[b], 0);
  r.kv = min(len, p.width << p.page_shift);
  r.before = len - r.n;
  r.tiles = ((r.n << p.g_shift) + ROWS - 1) / ROWS;
  return r;
}

// key blocks that row tile t has to look at: up to the last key that its last row sees
template <int ROWS>
__device__ __forceinline__ int paged_blocks(const PagedAttnParams& p, const PagedRequest& r, int t) {
  int keys = r.kv;
  if (p.causal && t + 1 < r.tiles)
    keys = min(keys, r.before + (((t + 1) * ROWS - 1) >> p.g_shift) + 1);
  return keys > 0 ? (keys - 1) / PG_BK + 1 : 1;   // a tile without keys still writes its rows
}

// units of a request
template <int ROWS>
__device__ __forceinline__ long long paged_units(const PagedAttnParams& p, const PagedRequest& r) {
  if (r.tiles == 0) return 0;
  if (!p.causal) return static_cast<long long>(r.tiles) * p.Hkv * paged_blocks<ROWS>(p, r, 0);
  long long u = 0;
  for (int t = 0; t < r.tiles; ++t) u += paged_blocks<ROWS>(p, r, t);
  return u * p.Hkv;
}

// A CTA's stretch of the line's `total` units, cut into ctas = min(N, total)
// stretches of q or q + 1 units (the first `more` of them), and the tile and
// block that it starts with.
struct PagedRange {
  int64_t total, q, left;      // left: units of this stretch
  PagedRequest r;              // request b
  int ctas, more;
  int b, tile, h, nb, kb0;
  int ord, tiles;              // number of the tile on the line; tiles of the call
};

// x / y and the rest; 64-bit division takes hundreds of cycles, and the numbers are nearly always small
__device__ __forceinline__ int64_t div64(int64_t x, int64_t y, int64_t& rest) {
  if ((x | y) >> 31 == 0) {
    const uint32_t d = static_cast<uint32_t>(x) / static_cast<uint32_t>(y);
    rest = x - static_cast<int64_t>(d) * y;
    return d;
  }
  const int64_t d = x / y;
  rest = x - d * y;
  return d;
}

// CTA whose stretch holds unit u
__device__ __forceinline__ int paged_holder(const PagedRange& g, int64_t u) {
  int64_t rest;
  const int64_t bound = g.more * (g.q + 1);
  return static_cast<int>(u < bound ? div64(u, g.q + 1, rest) : g.more + div64(u - bound, g.q, rest));
}

// One pass over the batch by the whole CTA: each thread sums the units of a
// run of requests, a scan gives their places on the line, and the thread that
// finds the stretch's start on its run tells the others.
template <int ROWS, int THREADS>
__device__ __forceinline__ PagedRange paged_range(const PagedAttnParams& p, int cta, int ctas) {
  constexpr int WARPS = THREADS / 32;
  __shared__ long long warp_sum[WARPS];
  __shared__ int warp_tiles[WARPS];
  __shared__ PagedRange found;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (p.batch + THREADS - 1) / THREADS;
  const int b0 = min(static_cast<int>(threadIdx.x) * per, p.batch), b1 = min(b0 + per, p.batch);
  long long sum = 0;
  int tiles = 0;
  PagedRequest r{};
  for (int b = b0; b < b1; ++b) {
    r = paged_request<ROWS>(p, b);
    sum += paged_units<ROWS>(p, r);
    tiles += r.tiles * p.Hkv;
  }
  long long upto = sum;
  int tiles_upto = tiles;
  if (__any_sync(0xffffffffu, sum > 0)) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, upto, o);
      const int y = __shfl_up_sync(0xffffffffu, tiles_upto, o);
      if (lane >= o) {
        upto += x;
        tiles_upto += y;
      }
    }
  }
  if (lane == 31) {
    warp_sum[warp] = upto;
    warp_tiles[warp] = tiles_upto;
  }
  if (threadIdx.x == 0) found.left = 0;   // nobody finds it if lengths change under the call
  __syncthreads();
  long long total = 0, before = 0;
  int tiles_all = 0, tiles_before = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w == warp) {
      before = total;
      tiles_before = tiles_all;
    }
    total += warp_sum[w];
    tiles_all += warp_tiles[w];
  }
  PagedRange g{};
  g.total = total;
  g.tiles = tiles_all;
  g.ctas = static_cast<int>(min64(ctas, total));
  if (cta >= g.ctas) return g;   // nothing to do (left = 0)
  int64_t rest;
  g.q = div64(total, g.ctas, rest);
  g.more = static_cast<int>(rest);
  g.left = g.q + (cta < g.more);
  const int64_t lo = g.q * cta + min(cta, g.more);
  long long at = before + upto - sum;
  if (lo >= at && lo < at + sum) {
    int tiles_at = tiles_before + tiles_upto - tiles, b = b0;
    if (per > 1) {
      for (;; ++b) {
        r = paged_request<ROWS>(p, b);
        const long long u = paged_units<ROWS>(p, r);
        if (lo < at + u || b + 1 == b1) break;
        at += u;
        tiles_at += r.tiles * p.Hkv;
      }
    }
    int64_t x = lo - at;         // units into request b
    g.r = r;
    g.b = b;
    g.nb = paged_blocks<ROWS>(p, r, 0);
    if (!p.causal) {
      g.tile = static_cast<int>(div64(x, static_cast<int64_t>(g.nb) * p.Hkv, x));
    } else {
      while (x >= static_cast<int64_t>(g.nb) * p.Hkv && g.tile + 1 < r.tiles) {
        x -= static_cast<int64_t>(g.nb) * p.Hkv;
        g.nb = paged_blocks<ROWS>(p, r, ++g.tile);
      }
    }
    g.h = static_cast<int>(div64(x, g.nb, x));
    g.kb0 = static_cast<int>(x);
    g.ord = tiles_at + g.tile * p.Hkv + g.h;
    found = g;
  }
  __syncthreads();
  return found;
}

// Walks the tiles of a stretch: the key blocks [kb0, kb1) of the nb of row
// tile `tile` of kv head h of request b.
template <int ROWS>
struct PagedWalk {
  PagedRequest r;
  int64_t left;
  int b, tile, h, nb, kb0, kb1;
  int ord;                     // number of the tile on the line

  __device__ __forceinline__ explicit PagedWalk(const PagedRange& g)
      : r(g.r), left(g.left), b(g.b), tile(g.tile), h(g.h), nb(g.nb), kb0(g.kb0),
        kb1(static_cast<int>(min64(g.nb, g.kb0 + g.left))), ord(g.ord) {}
  __device__ __forceinline__ bool more() const { return left > 0; }
  __device__ __forceinline__ bool whole() const { return kb0 == 0 && kb1 == nb; }
  __device__ __forceinline__ void next(const PagedAttnParams& p) {
    left -= kb1 - kb0;
    if (left <= 0) return;
    kb0 = 0;
    ++ord;
    if (++h == p.Hkv) {
      h = 0;
      if (++tile == r.tiles) {
        tile = 0;
        do {
          if (++b >= p.batch) {   // lengths that changed under the call
            left = 0;
            return;
          }
          r = paged_request<ROWS>(p, b);
        } while (r.tiles == 0);
      }
      nb = paged_blocks<ROWS>(p, r, tile);
    }
    kb1 = static_cast<int>(min64(nb, left));
  }
};

// where column c of row r of a partial slot lies: rows of floats, or for the
// 256-row tiles (a warp per 32 rows) [32 rows][D / 4][row] float4
template <int ROWS, int D>
__device__ __forceinline__ int64_t paged_part_at(int64_t slot, int r, int c) {
  return ROWS == 16 ? (slot * ROWS + r) * D + c
                    : (((slot * (ROWS / 32) + r / 32) * (D / 4) + c / 4) * 32 + r % 32) * 4 + c % 4;
}

// Lists tile number seg of a stretch for the merge kernel, if it begins there:
// with its pieces where the stretch does not finish it.  By tile, each has an
// entry; by CTA, only the last one of a stretch can be unfinished, and the
// caller writes `cut` in the end.
template <int ROWS>
__device__ __forceinline__ void paged_list(const PagedAttnParams& p, const PagedRange& g, const PagedWalk<ROWS>& w,
                                           int seg, PagedCut& cut) {
  cut = PagedCut{};
  cut.tiles = g.tiles;
  if (w.kb0 > 0) return;
  if (w.kb1 < w.nb) {
    cut.rows = min((w.r.n << p.g_shift) - w.tile * ROWS, ROWS);
    cut.t0 = w.r.t0;
    cut.row0 = w.tile * ROWS;
    cut.h = w.h;
    cut.first = blockIdx.x;
    cut.slot = 2 * blockIdx.x + (seg > 0);
    // the pieces behind this one are the first of each stretch up to the one that holds the tile's last unit
    const int c = blockIdx.x;
    const int64_t hi = g.q * (c + 1) + min(c + 1, g.more);
    cut.last = paged_holder(g, hi + (w.nb - w.kb1) - 1);
  }
  if (static_cast<uint32_t>(w.ord) < static_cast<uint32_t>(p.cuts_by_tile)) p.cuts[w.ord] = cut;
}

// A list by tile of a call without tiles: its first entry says so.
__device__ __forceinline__ void paged_list_none(const PagedAttnParams& p, const PagedRange& g) {
  if (g.tiles == 0 && p.cuts_by_tile && blockIdx.x == 0 && threadIdx.x == 0) p.cuts[0] = PagedCut{};
}

// A whole warp runs the code that issues tcgen05.mma or TMA copies, and one
// elected lane's instructions take effect: descriptors, addresses and
// coordinates then stay in uniform registers, where these instructions want
// them (taken one lane at a time an instruction costs 65 to 110 cycles).
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t is;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(is));
  return is;
}

__device__ __forceinline__ void tma_load_2d_lead(uint32_t lead, uint32_t smem_dst, const CUtensorMap* map, uint64_t* bar,
                                                 int x, int y, uint64_t policy) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %6, 0;\n\t"
      "@q cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4}], [%2], %5;\n\t}" ::"r"(smem_dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "l"(policy), "r"(lead)
      : "memory");
}

// Page ids of a request's row of the block table, 32 at a time, one per lane.
struct PagedIds {
  int first = -1, id = 0;
  // fetch what the pieces of a block from page `page` on need
  __device__ __forceinline__ void fetch(const PagedAttnParams& p, const int32_t* row, int page, int pieces) {
    if (first >= 0 && page + pieces <= first + 32) return;
    first = page;
    const int mine = page + static_cast<int>(threadIdx.x & 31);
    id = mine < p.width ? row[mine] : -1;
  }
  __device__ __forceinline__ int at(int page) const { return __shfl_sync(0xffffffffu, id, page - first); }
};

// The pages of a 64-key block: up to four pieces of `box` keys; their rows in
// the pools' tensor maps for kv head h, and which keys exist.
struct PagedBlock {
  int row[4];
  uint32_t good;               // pieces that lie in a page of the pool and below kv
  uint64_t valid;              // keys that do
};

__device__ __forceinline__ PagedBlock paged_block(const PagedAttnParams& p, const PagedIds& ids, int kb, int kv, int h,
                                                  int box, int piece_shift) {
  PagedBlock b;
  b.good = 0;
  b.valid = 0;
  const int first_page = (kb * PG_BK) >> p.page_shift;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i >> piece_shift) break;
    const int page = ids.at(first_page + i), key = kb * PG_BK + i * box;
    b.row[i] = page * (p.Hkv << p.page_shift) + (h << p.page_shift) + (key & ((1 << p.page_shift) - 1));
    if (page >= 0 && page < p.n_pages && key < kv) {
      b.good |= 1u << i;
      b.valid |= (box == 64 ? ~uint64_t(0) : ((uint64_t(1) << box) - 1)) << (i * box);
    }
  }
  const int keys = kv - kb * PG_BK;
  if (keys < PG_BK) b.valid &= keys > 0 ? (uint64_t(1) << keys) - 1 : 0;
  return b;
}

// the DK column boxes of the block's pieces into a stage of [column box][64 keys][64 columns]
template <int DK>
__device__ __forceinline__ void paged_fetch(uint32_t lead, const PagedBlock& b, const CUtensorMap* map, uint32_t stage,
                                            uint64_t* bar, int box, int piece_shift, uint64_t policy) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i >> piece_shift) break;
    if (!(b.good >> i & 1)) continue;
#pragma unroll
    for (int db = 0; db < DK; ++db)
      tma_load_2d_lead(lead, stage + db * PG_BK * 128 + i * box * 128, map, bar, db * 64, b.row[i], policy);
  }
}

// untiled copy of `bytes` (a multiple of 16; both addresses 16-byte aligned)
__device__ __forceinline__ void bulk_load(void* smem_dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(smem_dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// untiled store of `bytes` from shared memory (same rules), tracked by this thread's bulk-async group
__device__ __forceinline__ void bulk_store(void* dst, const void* smem_src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(smem_src)),
               "r"(bytes)
               : "memory");
}

// wait until every bulk store this thread committed is complete
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// c (16 x 8, fp32) += a (16 x 16) b (16 x 8), bf16
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// ----------------------------------------------------------------------------
// Few rows per request (single tokens): tiles of 16 packed rows (row = i * G +
// query head of the group), so that the G heads of a group share one read of
// their keys.
//
// Bound by HBM: 4 D bytes per key and kv head against 2 x 16 x 2 D operations,
// of which a token's G rows are useful.  So the products run on mma.sync
// (64 x 16 x 2 D x 2 per block, under a tenth of the block's time on the
// memory), and everything else serves the stream of pages: two producer
// warps keep STAGES blocks of K and V in flight, each landing swizzled by TMA
// so that ldmatrix reads it without bank conflicts; four warps take 16 of its
// 64 keys each, with running maxima, sums and rows of their own (no barrier
// between them inside a tile); at a tile's end they leave these in shared
// memory and go on, and a warp of its own joins them.
// One token for 64 requests of 256..8190 keys, 16/8 heads of 176: 234 us with
// the merge, 6.6 TB/s (1.0 of the copy peak); 33 requests of up to 1500 keys, 8/2
// heads of 128: 13.4 us; one request of 2048 keys: 9.5 us, of which the two blocks
// of a CTA are one.
// ----------------------------------------------------------------------------
constexpr int TOK_ROWS = 16;
constexpr int TOK_WARPS = 4;                       // consumer warps
constexpr int TOK_FIRST_CONSUMER = 2;              // warps 0 K, Q and descriptors, 1 V, 2..5 consumers, 6 join
constexpr int TOK_JOIN_WARP = TOK_FIRST_CONSUMER + TOK_WARPS;
constexpr int TOK_THREADS = 32 * (TOK_JOIN_WARP + 1);

template <int D>
struct TokCfg {
  static constexpr int DK = (D + 63) / 64;
  static constexpr int KV_BYTES = DK * PG_BK * 128;             // K or V of a block
  static constexpr int STAGES = D == 64 ? 6 : D == 128 ? 4 : 3;
  static constexpr int Q_LD = D * 2 + 16;                       // bytes of a query row: eight rows in different banks
  static constexpr int Q_BYTES = TOK_ROWS * Q_LD;
  static constexpr int Q_BUFS = STAGES + 1;                     // a tile's rows arrive with its first block
  static constexpr int O_LD = D + 4;
  static constexpr int O_BYTES = TOK_WARPS * TOK_ROWS * O_LD * 4;
  static constexpr int O_OFF = STAGES * 2 * KV_BYTES;
  static constexpr int Q_OFF = O_OFF + O_BYTES;
  static constexpr int TAIL_OFF = (Q_OFF + Q_BUFS * Q_BYTES + 127) / 128 * 128;
  static constexpr int SMEM = 1024 + TAIL_OFF + 1536;
};

enum TokFlags : int { TOK_FIRST = 1, TOK_LAST = 2, TOK_EXIT = 4, TOK_QBUF_SHIFT = 8 };

// what the consumers need to know of a stage
struct TokDesc {
  uint64_t valid;              // keys of the block in pages of the pool, below kv
  int flags;                   // TokFlags | buffer of the tile's queries << TOK_QBUF_SHIFT
  int n, kv, before;           // PagedRequest
  int row0;                    // first packed row of the tile
  int key0;                    // first key of the block
};

// (row, column) of a tile's live rows -> the output row
__device__ __forceinline__ int64_t paged_out_row(const PagedAttnParams& p, int t0, int packed, int h) {
  const int in_group = packed & ((1 << p.g_shift) - 1);
  return static_cast<int64_t>(t0 + (packed >> p.g_shift)) * p.Hq + (h << p.g_shift) + in_group;
}

// NaN in every row a stretch should have written (a wait ran out)
template <int ROWS, int D>
__device__ void paged_poison(const PagedAttnParams& p, const PagedRange& g) {
  int seg = 0;
  PagedCut cut{};
  cut.tiles = g.tiles;
  for (PagedWalk<ROWS> w(g); w.more(); w.next(p), ++seg) {
    paged_list<ROWS>(p, g, w, seg, cut);   // every thread writes the same
    const int live = min((w.r.n << p.g_shift) - w.tile * ROWS, ROWS);
    for (int i = threadIdx.x; i < live * D; i += blockDim.x) {
      const int64_t out = paged_out_row(p, w.r.t0, w.tile * ROWS + i / D, w.h);
      if (w.whole()) {
        p.o[out * D + i % D] = 0x7fc0;
        if (p.lse) p.lse[out] = NAN;
      } else {
        const int64_t slot = static_cast<int64_t>(blockIdx.x) * 2 + (seg > 0);
        p.part[paged_part_at<ROWS, D>(slot, i / D, i % D)] = NAN;
        p.part_ml[slot * ROWS + i / D] = make_float2(0.f, NAN);
      }
    }
  }
  if (threadIdx.x == 0 && !p.cuts_by_tile) p.cuts[blockIdx.x] = cut;
}

template <int D>
__global__ void __launch_bounds__(TOK_THREADS, 1) paged_token_kernel(const __grid_constant__ PagedAttnParams p) {
  using C = TokCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* s_o = reinterpret_cast<float*>(smem + C::O_OFF);       // [warp][16][O_LD]
  uint8_t* s_q = smem + C::Q_OFF;
  uint8_t* tail = smem + C::TAIL_OFF;
  uint64_t* full = reinterpret_cast<uint64_t*>(tail);
  uint64_t* empty = full + C::STAGES;
  uint64_t* o_full = empty + C::STAGES;                         // all four warps' rows of a tile written
  uint64_t* o_free = o_full + 1;                                // ... and joined
  TokDesc* desc = reinterpret_cast<TokDesc*>(tail + 256);       // [STAGES]
  float2* s_ml = reinterpret_cast<float2*>(tail + 768);         // [warp][16]
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tail + 1280);
  static_assert(C::STAGES * sizeof(TokDesc) <= 512 && (2 * C::STAGES + 2) * 8 <= 256, "tail layout");
  static_assert(TOK_WARPS * TOK_ROWS * sizeof(float2) == 512, "tail layout");

  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&p.k_map);
    tma_prefetch_desc(&p.v_map);
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 2);                  // both producers
      mbar_init(&empty[s], TOK_WARPS);
    }
    mbar_init(o_full, TOK_WARPS);
    mbar_init(o_free, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  pdl_wait();
  DG_TIMELINE_SCOPE(TLK_ATTENTION);
  const PagedRange g = paged_range<TOK_ROWS, TOK_THREADS>(p, blockIdx.x, gridDim.x);  // synchronises the CTA
  paged_list_none(p, g);
  bool ok = true;

  if (warp < TOK_FIRST_CONSUMER) {
    // ------------------ producers: warp 0 K, Q and descriptors, warp 1 V ------------------
    const bool is_k = warp == 0;
    const CUtensorMap* map = is_k ? &p.k_map : &p.v_map;
    const int box = min(1 << p.page_shift, PG_BK);              // keys per TMA box
    const int piece_shift = max(6 - p.page_shift, 0);           // 2^piece_shift pages (or part of one) per block
    const uint64_t pol = policy_evict_first();
    const uint32_t lead = elect_one();
    int it = 0, seg = 0;
    uint32_t issued = 0, par = 0;
    PagedCut cut{};
    for (PagedWalk<TOK_ROWS> w(g); ok && w.more(); w.next(p), ++seg) {
      if (!is_k && lane == 0) paged_list<TOK_ROWS>(p, g, w, seg, cut);
      const int32_t* tab = p.table + w.b * p.table_stride;
      const int live = min((w.r.n << p.g_shift) - w.tile * TOK_ROWS, TOK_ROWS);
      PagedIds ids;
      for (int kb = w.kb0; kb < w.kb1; ++kb, ++it) {
        const int s = it % C::STAGES;
        ids.fetch(p, tab, (kb * PG_BK) >> p.page_shift, 1 << piece_shift);
        const PagedBlock blk = paged_block(p, ids, kb, w.r.kv, w.h, box, piece_shift);
        ok = __all_sync(0xffffffffu, mbar_wait(&empty[s], ((it / C::STAGES) & 1) ^ 1, p.err) && !*abort_flag);
        if (!ok) break;
        const bool with_q = is_k && kb == w.kb0;
        if (lead) {
          if (is_k) {
            TokDesc d;
            d.valid = blk.valid;
            d.flags = (kb == w.kb0 ? TOK_FIRST : 0) | (kb + 1 == w.kb1 ? TOK_LAST : 0) |
                      (seg % C::Q_BUFS) << TOK_QBUF_SHIFT;
            d.n = w.r.n;
            d.kv = w.r.kv;
            d.before = w.r.before;
            d.row0 = w.tile * TOK_ROWS;
            d.key0 = kb * PG_BK;
            desc[s] = d;
          }
          mbar_arrive_expect_tx(&full[s], __popc(blk.good) * box * 128 * C::DK + (with_q ? live * D * 2 : 0));
        }
        __syncwarp();
        paged_fetch<C::DK>(lead, blk, map, smem_u32(smem) + s * 2 * C::KV_BYTES + (is_k ? 0 : C::KV_BYTES), &full[s],
                           box, piece_shift, pol);
        if (with_q && lane < live) {
          const int r = w.tile * TOK_ROWS + lane;
          bulk_load(s_q + (seg % C::Q_BUFS) * C::Q_BYTES + lane * C::Q_LD,
                    p.q + (w.r.t0 + (r >> p.g_shift)) * p.q_stride +
                        ((w.h << p.g_shift) + (r & ((1 << p.g_shift) - 1))) * D,
                    D * 2, &full[s]);
        }
        issued |= 1u << s;
        par = (par & ~(1u << s)) | (((it / C::STAGES) & 1) << s);
      }
    }
    if (lane == 0) {
      if (!is_k && !p.cuts_by_tile) p.cuts[blockIdx.x] = cut;
      const int s = it % C::STAGES;
      if (ok && mbar_wait(&empty[s], ((it / C::STAGES) & 1) ^ 1, p.err)) {
        if (is_k) desc[s].flags = TOK_EXIT;
        mbar_arrive(&full[s]);
      } else {
        *abort_flag = 1;
        // every copy issued here lands before the CTA exits
        for (int x = 0; x < C::STAGES; ++x)
          if (issued >> x & 1) mbar_wait(&full[x], par >> x & 1, p.err);
      }
    }
  } else if (warp < TOK_JOIN_WARP) {
    // ------------------------------- consumers ------------------------------
    const int w = warp - TOK_FIRST_CONSUMER, gr = lane >> 2, c = lane & 3, mi = lane >> 3, mr = lane & 7;
    uint32_t qf[D / 16][4];
    float o[D / 8][4];
    float m[2], l[2];
    int lim[2] = {0, 0};
    int seg = 0;
    for (int it = 0;; ++it) {
      const int s = it % C::STAGES;
      ok = __all_sync(0xffffffffu, mbar_wait(&full[s], (it / C::STAGES) & 1, p.err) && !*abort_flag);
      if (!ok) break;
      const TokDesc d = desc[s];
      if (d.flags & TOK_EXIT) break;
      const uint32_t k_at = smem_u32(smem + s * 2 * C::KV_BYTES), v_at = k_at + C::KV_BYTES;
      if (d.flags & TOK_FIRST) {
        const uint32_t q_at = smem_u32(s_q + (d.flags >> TOK_QBUF_SHIFT) * C::Q_BYTES);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          ldmatrix_x4(qf[kk], q_at + ((mi & 1) * 8 + mr) * C::Q_LD + kk * 32 + (mi >> 1) * 16);
#pragma unroll
        for (int t = 0; t < D / 8; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          m[x] = -INFINITY;
          l[x] = 0.f;
          lim[x] = p.causal ? min(d.kv, d.before + ((d.row0 + gr + 8 * x) >> p.g_shift) + 1) : d.kv;
        }
      }
      // S = Q K^T for this warp's 16 keys: two 16 x 8 tiles
      float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        uint32_t kf[4];
        ldmatrix_x4(kf, k_at + (kk >> 2) * (PG_BK * 128) + (w * 16 + (mi >> 1) * 8 + mr) * 128 +
                            ((((kk & 3) * 2 + (mi & 1)) ^ mr) << 4));
        mma_16816(sc[0], qf[kk], kf[0], kf[1]);
        mma_16816(sc[1], qf[kk], kf[2], kf[3]);
      }
      const uint32_t valid = static_cast<uint32_t>(d.valid >> (w * 16)) & 0xffffu;
      const int rel = d.key0 + w * 16;
      uint32_t pf[4];
      float f[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float mx = -INFINITY;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int key = t * 8 + 2 * c + e;
            float& v = sc[t][2 * x + e];
            v = (valid >> key & 1) && rel + key < lim[x] ? v * p.scale_log2 : -INFINITY;
            mx = fmaxf(mx, v);
          }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float mn = fmaxf(m[x], mx), base = mn == -INFINITY ? 0.f : mn;
        f[x] = ex2_approx(m[x] - base);
        m[x] = mn;
        float sum = 0.f;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          // p enters the second product in bf16 (off by up to 2^-8 of each, averaging out over keys); its sum stays fp32
          const float p0 = ex2_approx(sc[t][2 * x] - base), p1 = ex2_approx(sc[t][2 * x + 1] - base);
          sum += p0 + p1;
          pf[2 * t + x] = cvt_bf16x2(p0, p1);
        }
        l[x] = l[x] * f[x] + sum;
      }
      if (__any_sync(0xffffffffu, f[0] != 1.f || f[1] != 1.f)) {
#pragma unroll
        for (int t = 0; t < D / 8; ++t) {
          o[t][0] *= f[0];
          o[t][1] *= f[0];
          o[t][2] *= f[1];
          o[t][3] *= f[1];
        }
      }
      // O += P V; values of masked keys may be anything, so they are cleared
      const bool clear = valid != 0xffffu;
      const uint32_t keep0 = (valid >> (2 * c) & 1 ? 0xffffu : 0u) | (valid >> (2 * c + 1) & 1 ? 0xffff0000u : 0u);
      const uint32_t keep1 = (valid >> (2 * c + 8) & 1 ? 0xffffu : 0u) | (valid >> (2 * c + 9) & 1 ? 0xffff0000u : 0u);
#pragma unroll
      for (int t = 0; t < D / 16; ++t) {
        uint32_t vf[4];
        ldmatrix_x4_trans(vf, v_at + (t >> 2) * (PG_BK * 128) + (w * 16 + (mi & 1) * 8 + mr) * 128 +
                                  ((((t & 3) * 2 + (mi >> 1)) ^ mr) << 4));
        if (clear) {
          vf[0] &= keep0;
          vf[1] &= keep1;
          vf[2] &= keep0;
          vf[3] &= keep1;
        }
        mma_16816(o[2 * t], pf, vf[0], vf[1]);
        mma_16816(o[2 * t + 1], pf, vf[2], vf[3]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);
      if (!(d.flags & TOK_LAST)) continue;

      // -------- the tile's end: this warp's rows, once those of the tile before are joined --------
      const int live = min((d.n << p.g_shift) - d.row0, TOK_ROWS);
      if (seg > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(o_free, (seg - 1) & 1, p.err) && !*abort_flag);
        if (!ok) break;
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
        l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
        const int r = gr + 8 * x;
        if (r < live) {
          if (c == 0) s_ml[w * TOK_ROWS + r] = make_float2(m[x], l[x]);
          float* dst = s_o + (w * TOK_ROWS + r) * C::O_LD + 2 * c;
#pragma unroll
          for (int t = 0; t < D / 8; ++t) *reinterpret_cast<float2*>(dst + t * 8) = make_float2(o[t][2 * x], o[t][2 * x + 1]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(o_full);
      ++seg;
    }
    if (!ok) *abort_flag = 1;
  } else {
    // ---------------- join: the four warps' rows of a tile, in order ----------------
    int seg = 0;
    for (PagedWalk<TOK_ROWS> w(g); w.more(); w.next(p), ++seg) {
      ok = __all_sync(0xffffffffu, mbar_wait(o_full, seg & 1, p.err) && !*abort_flag);
      if (!ok) break;
      const int row0 = w.tile * TOK_ROWS, live = min((w.r.n << p.g_shift) - row0, TOK_ROWS);
      const bool whole = w.whole();
      const int64_t slot = static_cast<int64_t>(blockIdx.x) * 2 + (seg > 0);
#pragma unroll 2
      for (int i = lane; i < live * (D / 4); i += 32) {
        const int r = i / (D / 4), c4 = i % (D / 4) * 4;
        float M = -INFINITY;
#pragma unroll
        for (int x = 0; x < TOK_WARPS; ++x) M = fmaxf(M, s_ml[x * TOK_ROWS + r].x);
        const float base = M == -INFINITY ? 0.f : M;
        float L = 0.f;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int x = 0; x < TOK_WARPS; ++x) {
          const float2 ml = s_ml[x * TOK_ROWS + r];
          const float e = ex2_approx(ml.x - base);
          const float4 v = *reinterpret_cast<const float4*>(s_o + (x * TOK_ROWS + r) * C::O_LD + c4);
          L += e * ml.y;
          a.x += e * v.x;
          a.y += e * v.y;
          a.z += e * v.z;
          a.w += e * v.w;
        }
        if (whole) {
          const float inv = L == 0.f ? 0.f : 1.f / L;
          const int64_t row = paged_out_row(p, w.r.t0, row0 + r, w.h);
          *reinterpret_cast<uint2*>(p.o + row * D + c4) =
              make_uint2(cvt_bf16x2(a.x * inv, a.y * inv), cvt_bf16x2(a.z * inv, a.w * inv));
          if (p.lse && c4 == 0) p.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
        } else {
          *reinterpret_cast<float4*>(p.part + paged_part_at<TOK_ROWS, D>(slot, r, c4)) = a;
          if (c4 == 0) p.part_ml[slot * TOK_ROWS + r] = make_float2(M, L);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(o_free);
    }
    if (!ok) *abort_flag = 1;
  }
  __syncthreads();
  if (*abort_flag) paged_poison<TOK_ROWS, D>(p, g);
}

// ----------------------------------------------------------------------------
// Joins the tiles that the stretches cut, from the attention kernel's list:
//   o = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i,  M = max_i m_i
// over a tile's pieces, in one pass with a running maximum.  Bound by the
// latency of its loads, of which each thread keeps several in flight; a small
// tile's pieces are dealt out to groups of threads, joined in shared memory.
// 2.8 us behind a token kernel, 5 us for the 16 tiles of a canvas over 2k keys
// (26.7 MB of partial rows out of L2).
// ----------------------------------------------------------------------------
template <int ROWS>
struct MergeCfg {
  static constexpr int THREADS = ROWS == 16 ? 512 : 256;
  static constexpr int COLS = ROWS == 16 ? 1 : 2;    // groups of four columns of a thread
  static constexpr int DEEP = ROWS == 16 ? 8 : 5;    // pieces in flight
};

template <int COLS>
struct MergeAcc {
  float m = -INFINITY, l = 0.f;
  float4 o[COLS];
  __device__ __forceinline__ MergeAcc() {
#pragma unroll
    for (int k = 0; k < COLS; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __device__ __forceinline__ void add(float2 ml, const float4 (&v)[COLS]) {
    const float mn = fmaxf(m, ml.x), base = mn == -INFINITY ? 0.f : mn;
    const float e0 = ex2_approx(m - base), e1 = ex2_approx(ml.x - base);
    m = mn;
    l = l * e0 + ml.y * e1;
#pragma unroll
    for (int k = 0; k < COLS; ++k) {
      o[k].x = o[k].x * e0 + v[k].x * e1;
      o[k].y = o[k].y * e0 + v[k].y * e1;
      o[k].z = o[k].z * e0 + v[k].z * e1;
      o[k].w = o[k].w * e0 + v[k].w * e1;
    }
  }
};

template <int ROWS, int D>
__global__ void __launch_bounds__(MergeCfg<ROWS>::THREADS) paged_merge_kernel(const __grid_constant__ PagedAttnParams p) {
  using C = MergeCfg<ROWS>;
  __shared__ float4 s_o[ROWS == 16 ? C::THREADS : 1];
  __shared__ float2 s_ml[ROWS == 16 ? C::THREADS : 1];
  pdl_launch_dependents();
  pdl_wait();
  DG_TIMELINE_SCOPE(TLK_ATTN_MERGE);
  // by tile, the first entry says how many there are (both are fetched at once)
  const int tiles = p.cuts[0].tiles;
  const PagedCut cut = p.cuts[blockIdx.x];
  if ((p.cuts_by_tile && static_cast<int>(blockIdx.x) >= tiles) || cut.rows == 0) return;
  // items: a row's column group; neighbouring threads take columns of a row where rows lie whole, else rows
  const int items = ROWS == 16 ? cut.rows * (D / 4) : ROWS;
  const int groups = ROWS == 16 ? max(1, C::THREADS / items) : 1;
  const int grp = ROWS == 16 && groups > 1 ? threadIdx.x / items : 0;
  for (int i = threadIdx.x - grp * items; i < items; i += C::THREADS) {
    const int r = ROWS == 16 ? i / (D / 4) : i;
    const int c0 = ROWS == 16 ? i % (D / 4) * 4 : blockIdx.y * C::COLS * 4;
    if (r >= cut.rows || grp >= groups) break;
    MergeAcc<C::COLS> acc;
    for (int x0 = cut.first + grp; x0 <= cut.last; x0 += groups * C::DEEP) {
      float2 ml[C::DEEP];
      float4 v[C::DEEP][C::COLS];
#pragma unroll
      for (int y = 0; y < C::DEEP; ++y) {
        const int x = x0 + y * groups;
        if (x > cut.last) break;
        const int64_t slot = x == cut.first ? cut.slot : 2 * x;
        ml[y] = p.part_ml[slot * ROWS + r];
#pragma unroll
        for (int k = 0; k < C::COLS; ++k)
          v[y][k] = *reinterpret_cast<const float4*>(p.part + paged_part_at<ROWS, D>(slot, r, c0 + 4 * k));
      }
#pragma unroll
      for (int y = 0; y < C::DEEP; ++y) {
        if (x0 + y * groups > cut.last) break;
        acc.add(ml[y], v[y]);
      }
    }
    if (ROWS == 16 && groups > 1) {
      s_o[threadIdx.x] = acc.o[0];
      s_ml[threadIdx.x] = make_float2(acc.m, acc.l);
      break;   // one item per thread
    }
    const float inv = acc.l == 0.f ? 0.f : 1.f / acc.l;
    const int64_t row = paged_out_row(p, cut.t0, cut.row0 + r, cut.h);
#pragma unroll
    for (int k = 0; k < C::COLS; ++k)
      *reinterpret_cast<uint2*>(p.o + row * D + c0 + 4 * k) =
          make_uint2(cvt_bf16x2(acc.o[k].x * inv, acc.o[k].y * inv), cvt_bf16x2(acc.o[k].z * inv, acc.o[k].w * inv));
    if (p.lse && c0 == 0) p.lse[row] = acc.l == 0.f ? -INFINITY : (acc.m + log2f(acc.l)) * 0.69314718055994531f;
  }
  if (ROWS == 16 && groups > 1) {
    __syncthreads();
    const int i = threadIdx.x;
    if (i >= items) return;
    MergeAcc<1> acc;
    for (int x = 0; x < groups; ++x) {
      const float4 v[1] = {s_o[x * items + i]};
      acc.add(s_ml[x * items + i], v);
    }
    const int r = i / (D / 4), c0 = i % (D / 4) * 4;
    const float inv = acc.l == 0.f ? 0.f : 1.f / acc.l;
    const int64_t row = paged_out_row(p, cut.t0, cut.row0 + r, cut.h);
    *reinterpret_cast<uint2*>(p.o + row * D + c0) =
        make_uint2(cvt_bf16x2(acc.o[0].x * inv, acc.o[0].y * inv), cvt_bf16x2(acc.o[0].z * inv, acc.o[0].w * inv));
    if (p.lse && c0 == 0) p.lse[row] = acc.l == 0.f ? -INFINITY : (acc.m + log2f(acc.l)) * 0.69314718055994531f;
  }
}

}  // namespace dg
