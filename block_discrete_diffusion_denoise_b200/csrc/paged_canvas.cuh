// Paged attention for many rows per request (canvases, causal chunks): tiles
// of 256 packed rows (row = i * G + query head of the group) on tcgen05.
//
// A unit is 4 x 256 x 64 x D operations against 4 x 64 x D bytes of K and V, so
// the tensor core bounds it.  Two 128-row tiles of queries stay in shared
// memory and share every K and V block; S = Q K^T and O += P V go to TMEM
// (2 x 64 + 2 x D columns), one softmax thread per row.  Each query tile has an
// MMA warp of its own, which issues S(j) and then PV(j-1), so that a tile's
// softmax hides behind its next scores and the other tile's products.  (One
// warp for both tiles spent its time on the waits: 78 cycles for a barrier
// that is ready, 30 for a commit, 2800 for a unit.)  The warps are a
// persistent pipeline over the CTA's stretch of units (paged_attention.cuh);
// each role walks it by itself, and a word per unit tells the softmax warps
// which keys the producers found.  At D = 176 a unit's products take 1777
// cycles (48.6 per k-step of S, where both operands come from shared memory and
// Q is read again for each, 88.5 of P V) and a unit 2050 to 2100.  A canvas of
// 256 rows over 33,024 keys, 16/8 heads of 176: 96 us with the merge, 1000
// TFLOP/s (117 us once the power limit lowers the clock); eight canvases over
// 1.5k..6.5k keys 114 us; one over 2304 keys 21.8 us.
#pragma once

#include "paged_attention.cuh"

namespace dg {

constexpr int CV_TILE = 128;             // packed rows of a query tile (MMA M)
constexpr int CV_ROWS = 2 * CV_TILE;
constexpr int CV_MASKS = 8;               // ring of key masks, deeper than any role runs ahead
constexpr int CV_MMA_WARP = 2;           // warps 0 K, 1 V, 2 and 3 Q and MMA of tiles 0 and 1,
constexpr int CV_SOFTMAX_WARP = 4;       // 4..7 and 8..11 softmax of tiles 0 and 1
constexpr int CV_THREADS = 32 * (CV_SOFTMAX_WARP + 8);
constexpr float CV_RESCALE_LOG2 = 8.f;

template <int D>
struct CvCfg {
  static constexpr int DK = (D + 63) / 64;
  static constexpr int Q_BYTES = DK * CV_TILE * 128;
  static constexpr int KV_BYTES = DK * PG_BK * 128;
  static constexpr int P_BYTES = CV_TILE * PG_BK * 2;
  static constexpr int STAGES = D == 176 ? 2 : 4;          // of K and of V
  static constexpr int K_OFF = 2 * Q_BYTES;
  static constexpr int V_OFF = K_OFF + STAGES * KV_BYTES;
  static constexpr int P_OFF = V_OFF + STAGES * KV_BYTES;
  static constexpr int TAIL_OFF = P_OFF + 2 * P_BYTES;
  static constexpr int SMEM = 1024 + TAIL_OFF + 1024;
  static constexpr int S_COL = 0;                          // TMEM: S_q at q * 64, O_q at 128 + q * D
  static constexpr int O_COL = 2 * PG_BK;
  static constexpr int TMEM_COLS = O_COL + 2 * D <= 256 ? 256 : 512;
  static_assert(O_COL + 2 * D <= 512, "S and O accumulators must fit TMEM");
};

struct CanvasParams {
  PagedAttnParams a;
  CUtensorMap q_map;           // 4-D (D, G, Hkv, rows) over q; box (64, G, 1, 128 / G)
};

// Matrix descriptors of one operand that differ in their start address only:
// the low word carries it (16-byte units), the high word is the layout.
struct UmmaOperand {
  uint32_t lo, hi;
  __device__ __forceinline__ explicit UmmaOperand(uint64_t d)
      : lo(static_cast<uint32_t>(d)), hi(static_cast<uint32_t>(d >> 32)) {}
};

// D[tmem] (+)= A B^T with the operands' start addresses moved by a_off and b_off bytes
template <bool ACC>
__device__ __forceinline__ void umma_at(uint32_t lead, uint32_t tmem_d, const UmmaOperand& a, uint32_t a_off,
                                        const UmmaOperand& b, uint32_t b_off, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %2};\n\t"
      "mov.b64 db, {%3, %4};\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "setp.ne.b32 q, %7, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, p;\n\t}" ::"r"(tmem_d),
      "r"(a.lo + (a_off >> 4)), "r"(a.hi), "r"(b.lo + (b_off >> 4)), "r"(b.hi), "r"(idesc), "n"(ACC ? 1 : 0), "r"(lead)
      : "memory");
}

__device__ __forceinline__ void umma_commit_lead(uint32_t lead, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(lead)
      : "memory");
}

// mbar_wait by a whole warp with one answer
__device__ __forceinline__ bool mbar_wait_warp(uint64_t* bar, uint32_t parity, const DevErr& err) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const uint64_t t0 = globaltimer_ns();
  while (true) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if (__any_sync(0xffffffffu, globaltimer_ns() - t0 > err.limit_ns)) {
      raise_error(err, ERR_TIMEOUT);
      return false;
    }
  }
}

__device__ __forceinline__ uint64_t f32x2(float lo, float hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
__device__ __forceinline__ void f32x2_split(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t f32x2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t f32x2_add(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
template <int D>
__global__ void __launch_bounds__(CV_THREADS, 1) paged_canvas_kernel(const __grid_constant__ CanvasParams cp) {
  using C = CvCfg<D>;
  const PagedAttnParams& p = cp.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* tail = smem + C::TAIL_OFF;
  uint64_t* q_full = reinterpret_cast<uint64_t*>(tail);  // [2]
  uint64_t* k_full = q_full + 2;
  uint64_t* k_empty = k_full + C::STAGES;
  uint64_t* v_full = k_empty + C::STAGES;
  uint64_t* v_empty = v_full + C::STAGES;
  uint64_t* s_full = v_empty + C::STAGES;      // [2] MMA -> softmax q: scores ready, key mask written
  uint64_t* s_free = s_full + 2;               // [2] softmax q -> MMA: scores in registers
  uint64_t* p_full = s_free + 2;               // [2] softmax q -> MMA: P_q written
  uint64_t* o_done = p_full + 2;               // [2] MMA -> softmax q: O_q += P_q V complete
  uint64_t* o_free = o_done + 2;               // [2] softmax q -> MMA: O_q read at a tile's end
  uint64_t* drain = o_free + 2;                // [2]
  uint64_t* turn = drain + 2;                  // [2][4] warp w of the other warpgroup has left its exponentials
  uint64_t* key_mask = reinterpret_cast<uint64_t*>(tail + 512);  // [CV_MASKS] keys of the unit that exist
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(tail + 960);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tail + 964);
  static_assert((2 + 4 * C::STAGES + 20) * 8 <= 512 && CV_MASKS * 8 <= 448, "tail layout");
  static_assert(CV_MASKS >= C::STAGES + 4, "a mask is read before its slot comes round");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&p.k_map);
    tma_prefetch_desc(&p.v_map);
    tma_prefetch_desc(&cp.q_map);
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 2);               // both MMA warps
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 2);
    }
    for (int q = 0; q < 2; ++q) {
      mbar_init(&q_full[q], 1);
      mbar_init(&drain[q], 1);
      mbar_init(&s_full[q], 2);                // the products' commit, and the warp that has seen the mask
      mbar_init(&s_free[q], 4);                // a lane of each softmax warp
      mbar_init(&p_full[q], 4);
      mbar_init(&o_done[q], 1);
      mbar_init(&o_free[q], 4);
      for (int x = 0; x < 4; ++x) mbar_init(&turn[q * 4 + x], 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == CV_MMA_WARP) {
    tmem_alloc(tmem_holder, C::TMEM_COLS);
    tmem_relinquish();
    // Not before TMEM is this CTA's: a kernel that took it first and waits for this one would never get on.
    pdl_launch_dependents();
  }
  tc_fence_before();
  pdl_wait();
  DG_TIMELINE_SCOPE(TLK_ATTENTION);
  const PagedRange g = paged_range<CV_ROWS, CV_THREADS>(p, blockIdx.x, gridDim.x);  // synchronises the CTA
  paged_list_none(p, g);
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  bool ok = true;

  if (warp < 2) {
    // ----------------------- producers: warp 0 K, warp 1 V -----------------------
    const bool is_k = warp == 0;
    const CUtensorMap* map = is_k ? &p.k_map : &p.v_map;
    uint64_t* full = is_k ? k_full : v_full;
    uint64_t* empty = is_k ? k_empty : v_empty;
    uint8_t* ring = smem + (is_k ? C::K_OFF : C::V_OFF);
    const int box = min(1 << p.page_shift, PG_BK);              // keys per TMA box
    const int piece_shift = max(6 - p.page_shift, 0);           // 2^piece_shift pages (or part of one) per block
    const uint32_t lead = elect_one();
    const uint64_t pol = policy_evict_last();                   // the request's other row tiles read the block again
    int it = 0, seg = 0;
    uint32_t issued = 0, par = 0;
    PagedCut cut{};
    for (PagedWalk<CV_ROWS> w(g); ok && w.more(); w.next(p), ++seg) {
      if (!is_k && lane == 0) paged_list<CV_ROWS>(p, g, w, seg, cut);
      const int32_t* tab = p.table + w.b * p.table_stride;
      PagedIds ids;
      for (int kb = w.kb0; kb < w.kb1; ++kb, ++it) {
        const int s = it % C::STAGES;
        ids.fetch(p, tab, (kb * PG_BK) >> p.page_shift, 1 << piece_shift);
        const PagedBlock blk = paged_block(p, ids, kb, w.r.kv, w.h, box, piece_shift);
        ok = __all_sync(0xffffffffu, mbar_wait(&empty[s], ((it / C::STAGES) & 1) ^ 1, p.err) && !*abort_flag);
        if (!ok) break;
        if (lead) {
          // the mask's slot has been read by all: this K slot came free STAGES units behind its last user, and the
          // softmax of a tile is never more than two units behind its scores
          if (is_k) key_mask[it % CV_MASKS] = blk.valid;
          mbar_arrive_expect_tx(&full[s], __popc(blk.good) * box * 128 * C::DK);
        }
        __syncwarp();
        paged_fetch<C::DK>(lead, blk, map, smem_u32(ring) + s * C::KV_BYTES, &full[s], box, piece_shift, pol);
        issued |= 1u << s;
        par = (par & ~(1u << s)) | (((it / C::STAGES) & 1) << s);
      }
    }
    if (!ok) *abort_flag = 1;
    // every copy issued here lands before the CTA exits
    if (lane == 0) {
      for (int s = 0; s < C::STAGES; ++s)
        if (issued >> s & 1) mbar_wait(&full[s], par >> s & 1, p.err);
      if (!is_k && !p.cuts_by_tile) p.cuts[blockIdx.x] = cut;
    }
  } else if (warp < CV_SOFTMAX_WARP) {
    // ------------------- MMA issuer of tile q, and its queries -------------------
    constexpr uint32_t IDESC_S = umma_idesc_bf16(CV_TILE, PG_BK);             // Q, K both K-major
    constexpr uint32_t IDESC_PV = umma_idesc_bf16(CV_TILE, D) | (1u << 16);   // V is MN-major
    const uint32_t lead = elect_one();
    const uint32_t at = smem_u32(smem), tmem = __shfl_sync(0xffffffffu, tmem_base, 0);
    const int q = __shfl_sync(0xffffffffu, warp - CV_MMA_WARP, 0);
    UmmaOperand q_op(umma_desc_sw128(at)), p_op(umma_desc_sw128(at + C::P_OFF));
    q_op.lo += (q * C::Q_BYTES) >> 4;
    p_op.lo += (q * C::P_BYTES) >> 4;
    const UmmaOperand k_op(umma_desc_sw128(at + C::K_OFF)), v_op(umma_desc_sw128_mn(at + C::V_OFF, PG_BK * 128));
    int n = 0;                               // score tiles so far (P V is one behind)
    int held = 0;                            // row tiles so far that have used O
    int loads = 0;                           // row tiles so far whose queries were fetched
    // the queries of a row tile, into shared memory that no product reads any more
    auto fetch_q = [&](const PagedWalk<CV_ROWS>& w) {
      if (lead) mbar_arrive_expect_tx(&q_full[q], C::Q_BYTES);
      __syncwarp();
      if (lane < C::DK)
        tma_load_4d(smem + q * C::Q_BYTES + lane * CV_TILE * 128, &cp.q_map, &q_full[q], lane * 64, 0, w.h,
                    w.r.t0 + ((w.tile * CV_ROWS + q * CV_TILE) >> p.g_shift), policy_evict_last());
      ++loads;
    };
    auto has_rows = [&](const PagedWalk<CV_ROWS>& w) { return (w.r.n << p.g_shift) - w.tile * CV_ROWS > q * CV_TILE; };
    bool fetched = false;                    // this tile's queries are on their way
    int j = 0;
    for (PagedWalk<CV_ROWS> w(g); ok && w.more(); w.next(p)) {
      const int units = __shfl_sync(0xffffffffu, w.kb1 - w.kb0, 0);
      if (!__shfl_sync(0xffffffffu, has_rows(w), 0)) {
        // the other tile's blocks: pass them on
        for (int u = 0; ok && u < units; ++u, ++j) {
          const int st = j % C::STAGES, ph = (j / C::STAGES) & 1;
          ok = mbar_wait_warp(&k_full[st], ph, p.err);
          if (lead && ok) mbar_arrive(&k_empty[st]);
          ok = ok && mbar_wait_warp(&v_full[st], ph, p.err);
          if (lead && ok) mbar_arrive(&v_empty[st]);
        }
        continue;
      }
      if (!fetched) fetch_q(w);
      fetched = false;
      ok = mbar_wait_warp(&q_full[q], (loads - 1) & 1, p.err);
      // unit u's scores, then the product of unit u - 1
      for (int u = 0; ok && u <= units; ++u, ++j) {
        if (u < units) {
          const int ks = j % C::STAGES;
          ok = mbar_wait_warp(&k_full[ks], (j / C::STAGES) & 1, p.err) &&
               (n == 0 || mbar_wait_warp(&s_free[q], (n - 1) & 1, p.err));
          if (!ok) break;
          tc_fence_after();
          UmmaOperand b = k_op;
          b.lo += (ks * C::KV_BYTES) >> 4;
          const uint32_t d = tmem + C::S_COL + q * PG_BK;
          umma_at<false>(lead, d, q_op, 0, b, 0, IDESC_S);
#pragma unroll
          for (int kk = 1; kk < D / 16; ++kk)
            umma_at<true>(lead, d, q_op, (kk >> 2) * (CV_TILE * 128) + (kk & 3) * 32, b,
                          (kk >> 2) * (PG_BK * 128) + (kk & 3) * 32, IDESC_S);
          umma_commit_lead(lead, &s_full[q]);
          umma_commit_lead(lead, &k_empty[ks]);
          if (lead) mbar_arrive(&s_full[q]);
          ++n;
        }
        if (u == units - 1) {
          // the next row tile's queries, once the scores just issued are read
          PagedWalk<CV_ROWS> next = w;
          next.next(p);
          fetched = __shfl_sync(0xffffffffu, next.more() && has_rows(next), 0);
          if (fetched) {
            ok = mbar_wait_warp(&s_free[q], (n - 1) & 1, p.err);
            if (!ok) break;
            fetch_q(next);
          }
        }
        if (u > 0) {
          const int vs = (j - 1) % C::STAGES;
          const bool first = u == 1;
          const int i = n - 1 - (u < units);   // P of unit u - 1
          ok = mbar_wait_warp(&v_full[vs], ((j - 1) / C::STAGES) & 1, p.err) &&
               mbar_wait_warp(&p_full[q], i & 1, p.err) &&
               (!first || held == 0 || mbar_wait_warp(&o_free[q], (held - 1) & 1, p.err));
          if (!ok) break;
          tc_fence_after();
          UmmaOperand b = v_op;
          b.lo += (vs * C::KV_BYTES) >> 4;
          const uint32_t d = tmem + C::O_COL + q * D;
          if (first)
            umma_at<false>(lead, d, p_op, 0, b, 0, IDESC_PV);
          else
            umma_at<true>(lead, d, p_op, 0, b, 0, IDESC_PV);
#pragma unroll
          for (int kk = 1; kk < PG_BK / 16; ++kk) umma_at<true>(lead, d, p_op, kk * 32, b, kk * 2048, IDESC_PV);
          umma_commit_lead(lead, &o_done[q]);
          umma_commit_lead(lead, &v_empty[vs]);
        }
      }
      --j;
      ++held;
    }
    if (!ok) *abort_flag = 1;
    // every copy and MMA issued here has completed before shared memory and TMEM are released
    if (loads > 0) mbar_wait_warp(&q_full[q], (loads - 1) & 1, p.err);
    umma_commit_lead(lead, &drain[q]);
    mbar_wait_warp(&drain[q], 0, p.err);
  } else {
    // ----------------------- softmax warpgroup of tile wg -----------------------
    const int wg = (warp - CV_SOFTMAX_WARP) >> 2;
    const int quarter = warp & 3;                    // TMEM lanes this warp may access
    const int rloc = quarter * 32 + lane;            // row of the tile = TMEM lane
    const uint32_t t_row = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t s_col = t_row + C::S_COL + wg * PG_BK, o_col = t_row + C::O_COL + wg * D;
    uint8_t* pdst = smem + C::P_OFF + wg * C::P_BYTES + rloc * 128;
    int j = 0, seg = 0, n_s = 0;                     // units of the stretch, tiles, score tiles read so far
    int turns = 0;                                   // units so far that both tiles had rows in
    for (PagedWalk<CV_ROWS> w(g); ok && w.more(); w.next(p), ++seg) {
      const int row0 = w.tile * CV_ROWS, units = w.kb1 - w.kb0;
      if ((w.r.n << p.g_shift) - row0 <= wg * CV_TILE) {        // no live row in this tile
        j += units;
        continue;
      }
      const bool both = (w.r.n << p.g_shift) - row0 > CV_TILE;
      const int r = row0 + wg * CV_TILE + rloc;      // packed row of the request
      const bool live = r < (w.r.n << p.g_shift);
      // keys [0, lim) are this row's
      const int lim = !live ? 0 : p.causal ? min(w.r.kv, w.r.before + (r >> p.g_shift) + 1) : w.r.kv;
      const int lim_all = __reduce_min_sync(0xffffffffu, live ? lim : INT32_MAX);
      float mref = -INFINITY, lsum = 0.f;
      for (int u = 0; u < units; ++u, ++j, ++n_s) {
        const int key0 = (w.kb0 + u) * PG_BK;
        // warp-uniform decisions: tcgen05.ld below is a warp-collective
        ok = __all_sync(0xffffffffu, mbar_wait(&s_full[wg], n_s & 1, p.err));
        if (!ok) break;
        const uint64_t valid = key_mask[j % CV_MASKS];
        tc_fence_after();
        float s[PG_BK];
        tmem_ld64(s_col, s);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_free[wg]);
        if (key0 + PG_BK > lim_all || valid != ~uint64_t(0)) {
          const int lj = lim - key0;
          const uint64_t seen = lj >= PG_BK ? valid : lj <= 0 ? 0 : valid & ((uint64_t(1) << lj) - 1);
          const uint32_t half[2] = {static_cast<uint32_t>(seen), static_cast<uint32_t>(seen >> 32)};
#pragma unroll
          for (int c = 0; c < PG_BK; ++c)
            if (!(half[c / 32] & (1u << (c % 32)))) s[c] = -INFINITY;
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < PG_BK; c += 2) mx[(c >> 1) & 3] = fmaxf(mx[(c >> 1) & 3], fmaxf(s[c], s[c + 1]));
        // scale > 0, so the maximum of the scaled scores is the scaled maximum
        const float mblk = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2;
        // P = 2^(s - mref); the reference is raised only when a block passes it by 2^8, so that rescaling O is rare
        const bool resc = mblk > mref + CV_RESCALE_LOG2;          // false while nothing is visible
        const float factor = resc ? ex2_approx(mref - mblk) : 1.f;  // 0 when mref = -inf
        if (resc) mref = mblk;
        const float base = mref == -INFINITY ? 0.f : mref;
        if (u > 0) {
          // O_q += P_q V of the unit before has completed: O_q is stable and P_q's buffer free
          ok = __all_sync(0xffffffffu, mbar_wait(&o_done[wg], (n_s - 1) & 1, p.err));
          if (!ok) break;
          tc_fence_after();
          if (__any_sync(0xffffffffu, resc)) {
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 16) {
              float v[16];
              tmem_ld16(o_col + c0, v);
#pragma unroll
              for (int e = 0; e < 16; ++e) v[e] *= factor;
              tmem_st16(o_col + c0, v);
            }
            tmem_st_wait();
          }
        }
        if (valid != ~uint64_t(0)) {
          // values of masked keys may be anything, and 0 * NaN is NaN: they are cleared (by both warpgroups, each
          // before its own product) in the swizzled rows of the V block
          ok = __all_sync(0xffffffffu, mbar_wait(&v_full[j % C::STAGES], (j / C::STAGES) & 1, p.err));
          if (!ok) break;
          uint8_t* vb = smem + C::V_OFF + (j % C::STAGES) * C::KV_BYTES;
          for (int i = rloc; i < PG_BK * 8; i += CV_TILE)
            if (!(valid >> (i / 8) & 1)) {
#pragma unroll
              for (int b = 0; b < C::DK; ++b) reinterpret_cast<uint4*>(vb + b * PG_BK * 128)[i] = make_uint4(0, 0, 0, 0);
            }
        }
        const uint64_t scale2 = f32x2(p.scale_log2, p.scale_log2), base2 = f32x2(-base, -base);
        // The two warps of an SM quarter take turns at the exponentials, tile 0 first: without that they fall into
        // step, share the MUFU at half speed and leave it and the tensor core idle together (2550 cycles a unit).
        if (both) ok = mbar_wait(&turn[wg * 4 + quarter], (turns & 1) ^ (wg == 0), p.err);
        uint64_t l2[2] = {0, 0};
#pragma unroll
        for (int ch = 0; ch < 8; ++ch) {
          uint32_t pk[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            // p enters the second product in bf16 (off by up to 2^-8 of each, averaging out over keys); its sum stays fp32
            float x0, x1;
            f32x2_split(f32x2_fma(f32x2(s[8 * ch + 2 * c], s[8 * ch + 2 * c + 1]), scale2, base2), x0, x1);
            const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
            l2[c & 1] = f32x2_add(l2[c & 1], f32x2(p0, p1));
            pk[c] = cvt_bf16x2(p0, p1);
          }
          // row rloc of a K-major 128-byte-swizzled tile: 16-byte chunk c lands at c ^ (row & 7)
          *reinterpret_cast<uint4*>(pdst + ((ch ^ (rloc & 7)) << 4)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
        }
        if (both) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&turn[(wg ^ 1) * 4 + quarter]);
          ++turns;
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[wg]);
        float l0, l1;
        f32x2_split(f32x2_add(l2[0], l2[1]), l0, l1);
        lsum = lsum * factor + (l0 + l1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
      }
      if (!ok) break;

      // ------------- the tile's end: its rows, or their partial slot -------------
      ok = __all_sync(0xffffffffu, ok && mbar_wait(&o_done[wg], (n_s - 1) & 1, p.err));
      if (!ok) break;
      tc_fence_after();
      const bool whole = w.whole();
      const float inv = lsum == 0.f ? 0.f : 1.f / lsum;
      const int64_t row = live ? paged_out_row(p, w.r.t0, r, w.h) : 0;
      const int64_t slot = static_cast<int64_t>(blockIdx.x) * 2 + (seg > 0);
      if (whole) {
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 16) {
          float v[16];
          tmem_ld16(o_col + c0, v);
          if (!live) continue;
          uint4* dst = reinterpret_cast<uint4*>(p.o + row * D + c0);
#pragma unroll
          for (int e = 0; e < 16; e += 8)
            dst[e / 8] = make_uint4(cvt_bf16x2(v[e] * inv, v[e + 1] * inv), cvt_bf16x2(v[e + 2] * inv, v[e + 3] * inv),
                                    cvt_bf16x2(v[e + 4] * inv, v[e + 5] * inv), cvt_bf16x2(v[e + 6] * inv, v[e + 7] * inv));
        }
      } else {
        // A warp's 32 rows go out in bulk copies of 32 columns through its rows of the P buffer, which is free now.
        float4* stage = reinterpret_cast<float4*>(smem + C::P_OFF + wg * C::P_BYTES + quarter * 4096) + lane;
        float* dst = p.part + paged_part_at<CV_ROWS, D>(slot, wg * CV_TILE + quarter * 32, 0);
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 32) {
          const bool wide = c0 + 32 <= D;      // D is a multiple of 16
          if (lane == 0) bulk_wait_read_all();
          __syncwarp();
          auto put = [&](auto& v) {
            constexpr int N = sizeof(v) / sizeof(float);
#pragma unroll
            for (int e = 0; e < N; e += 4) stage[e / 4 * 32] = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
          };
          if (wide) {
            float v[32];
            tmem_ld32(o_col + c0, v);
            put(v);
          } else {
            float v[16];
            tmem_ld16(o_col + c0, v);
            put(v);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            bulk_store(dst + c0 * 32, stage, (wide ? 32 : 16) * 128);
            bulk_commit_group();
          }
        }
        if (lane == 0) bulk_wait_read_all();
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&o_free[wg]);
      if (live) {
        if (!whole)
          p.part_ml[slot * CV_ROWS + wg * CV_TILE + rloc] = make_float2(mref, lsum);
        else if (p.lse)
          p.lse[row] = lsum == 0.f ? -INFINITY : (mref + log2f(lsum)) * 0.69314718055994531f;
      }
    }
    if (lane == 0) bulk_wait_all();
    if (!ok) *abort_flag = 1;
  }
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) paged_poison<CV_ROWS, D>(p, g);
  if (warp == CV_MMA_WARP) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

}  // namespace dg
