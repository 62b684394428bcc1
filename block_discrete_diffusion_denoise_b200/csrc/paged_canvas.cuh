// Paged attention for many rows per request (canvases, causal chunks): tiles
// of 256 packed rows (row = i * G + query head of the group) on tcgen05.
//
// A unit is 4 x 256 x 64 x D operations against 4 x 64 x D bytes of K and V, so
// the tensor core bounds it.  Two 128-row tiles of queries stay in shared
// memory and share every K and V block; S = Q K^T and O += P V go to TMEM
// (2 x 64 + 2 x D columns), one softmax thread per row.  In the steady state
// the tensor core runs
//   S_0(j) PV_0(j-1) S_1(j) PV_1(j-1) S_0(j+1) ...
// so that a tile's softmax has the other tile's products and its own next
// scores to hide behind.  The warps are a persistent pipeline over the CTA's
// stretch of units (paged_attention.cuh): a descriptor per unit, in a ring of
// its own, tells the MMA and softmax warps what the producers fetched.
#pragma once

#include "paged_attention.cuh"

namespace dg {

constexpr int CV_TILE = 128;             // packed rows of a query tile (MMA M)
constexpr int CV_ROWS = 2 * CV_TILE;
constexpr int CV_DESCS = 8;
constexpr int CV_SOFTMAX_WARP = 3;       // warps 0 K and Q, 1 V, 2 MMA, 3..6 and 7..10 softmax of tiles 0 and 1
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

// what the MMA and softmax warps need to know of a unit
struct CvDesc {
  uint64_t valid;              // keys of the block in pages of the pool, below kv
  int flags, nq;               // query tiles with live rows
  int t0, n, kv, h;
  int row0;                    // first packed row of the tile
  int key0;                    // first key of the block
};

template <int D>
__global__ void __launch_bounds__(CV_THREADS, 1) paged_canvas_kernel(const __grid_constant__ CanvasParams cp) {
  DG_TIMELINE_SCOPE(TLK_ATTENTION);
  using C = CvCfg<D>;
  const PagedAttnParams& p = cp.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* tail = smem + C::TAIL_OFF;
  uint64_t* q_full = reinterpret_cast<uint64_t*>(tail);
  uint64_t* q_empty = q_full + 1;
  uint64_t* k_full = q_full + 2;
  uint64_t* k_empty = k_full + C::STAGES;
  uint64_t* v_full = k_empty + C::STAGES;
  uint64_t* v_empty = v_full + C::STAGES;
  uint64_t* d_full = v_empty + C::STAGES;      // [CV_DESCS] K producer -> MMA and softmax: descriptor written
  uint64_t* d_empty = d_full + CV_DESCS;       // [CV_DESCS] ... and read
  uint64_t* s_full = d_empty + CV_DESCS;       // [2] MMA -> softmax q: scores ready
  uint64_t* s_free = s_full + 2;               // [2] softmax q -> MMA: scores in registers
  uint64_t* p_full = s_free + 2;               // [2] softmax q -> MMA: P_q written
  uint64_t* o_done = p_full + 2;               // [2] MMA -> softmax q: O_q += P_q V complete
  uint64_t* o_free = o_done + 2;               // [2] softmax q -> MMA: O_q read at a tile's end
  uint64_t* drain = o_free + 2;
  CvDesc* desc = reinterpret_cast<CvDesc*>(tail + 512);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(tail + 960);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tail + 964);
  static_assert((2 + 4 * C::STAGES + 2 * CV_DESCS + 11) * 8 <= 512, "tail layout");
  static_assert(CV_DESCS * sizeof(CvDesc) <= 448, "tail layout");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&p.k_map);
    tma_prefetch_desc(&p.v_map);
    tma_prefetch_desc(&cp.q_map);
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    for (int s = 0; s < CV_DESCS; ++s) {
      mbar_init(&d_full[s], 1);
      mbar_init(&d_empty[s], 9);               // the MMA thread and eight softmax warps
    }
    for (int q = 0; q < 2; ++q) {
      mbar_init(&s_full[q], 1);
      mbar_init(&s_free[q], CV_TILE);
      mbar_init(&p_full[q], CV_TILE);
      mbar_init(&o_done[q], 1);
      mbar_init(&o_free[q], CV_TILE);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 2) {
    tmem_alloc(tmem_holder, C::TMEM_COLS);
    tmem_relinquish();
  }
  pdl_launch_dependents();
  tc_fence_before();
  const PagedRange g = paged_range<CV_ROWS>(p, blockIdx.x, gridDim.x);  // synchronises the CTA
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  const int G = p.Hq / p.Hkv;
  bool ok = true;

  if (warp < 2) {
    // -------------------- producers: warp 0 Q and K, warp 1 V --------------------
    const bool is_k = warp == 0;
    const CUtensorMap* map = is_k ? &p.k_map : &p.v_map;
    uint64_t* full = is_k ? k_full : v_full;
    uint64_t* empty = is_k ? k_empty : v_empty;
    uint8_t* ring = smem + (is_k ? C::K_OFF : C::V_OFF);
    const int box = min(1 << p.page_shift, PG_BK);              // keys per TMA box
    const int pieces = PG_BK / box;                             // pages (or part of one) per block
    const int rows_per_page = p.Hkv << p.page_shift;
    const int my_piece = lane % pieces, db = lane / pieces;     // box of this lane
    const uint64_t pol = policy_evict_last();                   // the request's other row tiles read the block again
    int it = 0, seg = 0;
    uint32_t issued = 0, par = 0;
    for (PagedWalk<CV_ROWS> w(p, g); ok && w.more(); w.next(p), ++seg) {
      const int32_t* tab = p.table + w.b * p.table_stride;
      const int row0 = w.tile * CV_ROWS;
      const int nq = w.r.n * G - row0 > CV_TILE ? 2 : 1;
      if (is_k) {
        ok = __all_sync(0xffffffffu, (seg == 0 || mbar_wait(q_empty, (seg - 1) & 1, p.err)) && !*abort_flag);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(q_full, nq * C::Q_BYTES);
        __syncwarp();
        if (lane < nq * C::DK) {
          const int q = lane / C::DK, b = lane % C::DK;
          tma_load_4d(smem + q * C::Q_BYTES + b * CV_TILE * 128, &cp.q_map, q_full, b * 64, 0, w.h,
                      w.r.t0 + (row0 + q * CV_TILE) / G, pol);
        }
      }
      int ids0 = -1, ids = 0;                                   // page ids [ids0, ids0 + 32) of the request, one per lane
      for (int kb = w.kb0; kb < w.kb1; ++kb, ++it) {
        const int s = it % C::STAGES;
        const int first_page = (kb * PG_BK) >> p.page_shift;
        if (ids0 < 0 || first_page + pieces > ids0 + 32) {
          ids0 = first_page;
          ids = ids0 + lane < p.width ? tab[ids0 + lane] : -1;
        }
        const int page = __shfl_sync(0xffffffffu, ids, first_page + my_piece - ids0);
        const int key = kb * PG_BK + my_piece * box;
        const bool good = page >= 0 && page < p.n_pages && key < w.r.kv;
        const uint32_t pmask = __ballot_sync(0xffffffffu, good && lane < pieces);
        ok = __all_sync(0xffffffffu, mbar_wait(&empty[s], ((it / C::STAGES) & 1) ^ 1, p.err) &&
                                         (!is_k || mbar_wait(&d_empty[it % CV_DESCS], ((it / CV_DESCS) & 1) ^ 1, p.err)) &&
                                         !*abort_flag);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&full[s], __popc(pmask) * box * 128 * C::DK);
          if (is_k) {
            uint64_t valid = 0;
            for (int i = 0; i < pieces; ++i)
              if (pmask >> i & 1) valid |= (box == 64 ? ~uint64_t(0) : ((uint64_t(1) << box) - 1)) << (i * box);
            const int keys = w.r.kv - kb * PG_BK;
            if (keys < PG_BK) valid &= keys > 0 ? (uint64_t(1) << keys) - 1 : 0;
            CvDesc d;
            d.valid = valid;
            d.flags = (kb == w.kb0 ? TOK_FIRST : 0) | (kb + 1 == w.kb1 ? TOK_LAST : 0) | (w.whole() ? TOK_WHOLE : 0) |
                      (seg > 0 ? TOK_SLOT1 : 0);
            d.nq = nq;
            d.t0 = w.r.t0;
            d.n = w.r.n;
            d.kv = w.r.kv;
            d.h = w.h;
            d.row0 = row0;
            d.key0 = kb * PG_BK;
            desc[it % CV_DESCS] = d;
            mbar_arrive(&d_full[it % CV_DESCS]);
          }
        }
        __syncwarp();
        if (db < C::DK && good)
          tma_load_2d(ring + s * C::KV_BYTES + db * PG_BK * 128 + my_piece * box * 128, map, &full[s], db * 64,
                      page * rows_per_page + (w.h << p.page_shift) + (key & ((1 << p.page_shift) - 1)), pol);
        issued |= 1u << s;
        par = (par & ~(1u << s)) | (((it / C::STAGES) & 1) << s);
      }
    }
    if (is_k && ok && lane == 0) {
      ok = mbar_wait(&d_empty[it % CV_DESCS], ((it / CV_DESCS) & 1) ^ 1, p.err);
      if (ok) {
        desc[it % CV_DESCS].flags = TOK_EXIT;
        mbar_arrive(&d_full[it % CV_DESCS]);
      }
    }
    if (!ok) *abort_flag = 1;
    // every copy issued here lands before the CTA exits
    if (lane == 0) {
      for (int s = 0; s < C::STAGES; ++s)
        if (issued >> s & 1) mbar_wait(&full[s], par >> s & 1, p.err);
      if (is_k && seg > 0 && !ok) mbar_wait(q_full, (seg - 1) & 1, p.err);
    }
  } else if (warp == 2) {
    // -------------------------------- MMA issuer --------------------------------
    if (lane == 0) {
      constexpr uint32_t IDESC_S = umma_idesc_bf16(CV_TILE, PG_BK);             // Q, K both K-major
      constexpr uint32_t IDESC_PV = umma_idesc_bf16(CV_TILE, D) | (1u << 16);   // V is MN-major
      const uint32_t q_addr = smem_u32(smem), k_addr = q_addr + C::K_OFF, v_addr = q_addr + C::V_OFF,
                     p_addr = q_addr + C::P_OFF;
      int cs[2] = {0, 0}, cpv[2] = {0, 0};     // score and P V products of each tile so far
      int used[2] = {0, 0};                    // tiles that have held O_q
      int seg = 0;
      // O_q += P_q V of unit j (acc: not the tile's first)
      auto pv = [&](int q, int j, bool acc) {
        if (!mbar_wait(&p_full[q], cpv[q] & 1, p.err)) return false;
        if (!acc && used[q] > 0 && !mbar_wait(&o_free[q], (used[q] - 1) & 1, p.err)) return false;
        if (!acc) ++used[q];
        tc_fence_after();
        const uint32_t vb = v_addr + (j % C::STAGES) * C::KV_BYTES, pb = p_addr + q * C::P_BYTES;
#pragma unroll
        for (int kk = 0; kk < PG_BK / 16; ++kk)
          umma_bf16(tmem_base + C::O_COL + q * D, umma_desc_sw128(pb + kk * 32),
                    umma_desc_sw128_mn(vb + kk * 2048, PG_BK * 128), IDESC_PV, (acc || kk > 0) ? 1u : 0u);
        umma_commit(&o_done[q]);
        ++cpv[q];
        return true;
      };
      bool prev_first = false;
      for (int j = 0; ok; ++j) {
        const int ds = j % CV_DESCS, ks = j % C::STAGES;
        ok = mbar_wait(&d_full[ds], (j / CV_DESCS) & 1, p.err) && !*abort_flag;
        if (!ok) break;
        const int flags = desc[ds].flags, nq = desc[ds].nq;
        if (flags & TOK_EXIT) break;
        mbar_arrive(&d_empty[ds]);
        const bool first = flags & TOK_FIRST;
        ok = (!first || mbar_wait(q_full, seg & 1, p.err)) && mbar_wait(&k_full[ks], (j / C::STAGES) & 1, p.err);
        for (int q = 0; q < nq && ok; ++q) {
          if (cs[q] > 0) ok = mbar_wait(&s_free[q], (cs[q] - 1) & 1, p.err);
          if (!ok) break;
          tc_fence_after();
          const uint32_t kb = k_addr + ks * C::KV_BYTES, qb = q_addr + q * C::Q_BYTES;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            umma_bf16(tmem_base + C::S_COL + q * PG_BK, umma_desc_sw128(qb + (kk >> 2) * (CV_TILE * 128) + (kk & 3) * 32),
                      umma_desc_sw128(kb + (kk >> 2) * (PG_BK * 128) + (kk & 3) * 32), IDESC_S, kk > 0 ? 1u : 0u);
          umma_commit(&s_full[q]);
          ++cs[q];
          if (q == nq - 1) umma_commit(&k_empty[ks]);
          if (!first) {
            if (q == 0) ok = mbar_wait(&v_full[(j - 1) % C::STAGES], ((j - 1) / C::STAGES) & 1, p.err);
            ok = ok && pv(q, j - 1, !prev_first);
            if (ok && q == nq - 1) umma_commit(&v_empty[(j - 1) % C::STAGES]);
          }
        }
        if (ok && (flags & TOK_LAST)) {
          umma_commit(q_empty);
          ok = mbar_wait(&v_full[ks], (j / C::STAGES) & 1, p.err);
          for (int q = 0; q < nq && ok; ++q) ok = pv(q, j, !first);
          if (ok) umma_commit(&v_empty[ks]);
          ++seg;
        }
        prev_first = first;
      }
      if (!ok) *abort_flag = 1;
      // every MMA issued has completed before TMEM or its operands are released
      umma_commit(drain);
      mbar_wait(drain, 0, p.err);
    }
  } else {
    // ----------------------- softmax warpgroup of tile wg -----------------------
    const int wg = (warp - CV_SOFTMAX_WARP) >> 2;
    const int quarter = warp & 3;                    // TMEM lanes this warp may access
    const int rloc = quarter * 32 + lane;            // row of the tile = TMEM lane
    const uint32_t t_row = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t s_col = t_row + C::S_COL + wg * PG_BK, o_col = t_row + C::O_COL + wg * D;
    uint8_t* pdst = smem + C::P_OFF + wg * C::P_BYTES + rloc * 128;
    float mref = -INFINITY, lsum = 0.f;
    int lim = 0;                                     // keys [0, lim) are this row's
    int n_s = 0;                                     // score tiles read so far
    for (int j = 0;; ++j) {
      const int ds = j % CV_DESCS;
      // warp-uniform decisions: tcgen05.ld below is a warp-collective
      ok = __all_sync(0xffffffffu, mbar_wait(&d_full[ds], (j / CV_DESCS) & 1, p.err) && !*abort_flag);
      if (!ok) break;
      const CvDesc d = desc[ds];
      if (d.flags & TOK_EXIT) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(&d_empty[ds]);
      if (wg >= d.nq) continue;
      const int r = d.row0 + wg * CV_TILE + rloc;    // packed row of the request
      const bool live = r < d.n * G;
      const bool first = d.flags & TOK_FIRST;
      if (first) {
        mref = -INFINITY;
        lsum = 0.f;
        lim = !live ? 0 : p.causal ? min(d.kv, d.kv - d.n + r / G + 1) : d.kv;
      }
      ok = __all_sync(0xffffffffu, mbar_wait(&s_full[wg], n_s & 1, p.err) && !*abort_flag);
      if (!ok) break;
      tc_fence_after();
      float s[64];
      tmem_ld64(s_col, s);
      tc_fence_before();
      mbar_arrive(&s_free[wg]);
      const bool full = __all_sync(0xffffffffu, !live || lim - d.key0 >= PG_BK) && d.valid == ~uint64_t(0);
      if (!full) {
        const int lj = lim - d.key0;
#pragma unroll
        for (int c = 0; c < PG_BK; ++c)
          if (c >= lj || !(d.valid >> c & 1)) s[c] = -INFINITY;
      }
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int c = 0; c < PG_BK; ++c) mx[c & 3] = fmaxf(mx[c & 3], s[c]);
      // scale > 0, so the maximum of the scaled scores is the scaled maximum
      const float mblk = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2;
      // P = 2^(s - mref); the reference is raised only when a block passes it by 2^8, so that rescaling O is rare
      const bool resc = mblk > mref + CV_RESCALE_LOG2;          // false while nothing is visible
      const float factor = resc ? ex2_approx(mref - mblk) : 1.f;  // 0 when mref = -inf
      if (resc) mref = mblk;
      const float base = mref == -INFINITY ? 0.f : mref;
      lsum *= factor;
      float l = 0.f;
      uint32_t pk[PG_BK / 2];
#pragma unroll
      for (int c = 0; c < PG_BK / 2; ++c) {
        // p enters the second product in bf16 (2^-9 of each, averaging out over keys); its sum stays fp32
        const float p0 = ex2_approx(fmaf(s[2 * c], p.scale_log2, -base));
        const float p1 = ex2_approx(fmaf(s[2 * c + 1], p.scale_log2, -base));
        l += p0 + p1;
        pk[c] = pack_bf16x2(p0, p1);
      }
      lsum += l;
      if (!first) {
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
      if (d.valid != ~uint64_t(0)) {
        // values of masked keys may be anything, and 0 * NaN is NaN: they are cleared (by both warpgroups, each
        // before its own product) in the swizzled rows of the V block
        ok = __all_sync(0xffffffffu, mbar_wait(&v_full[j % C::STAGES], (j / C::STAGES) & 1, p.err));
        if (!ok) break;
        uint8_t* vb = smem + C::V_OFF + (j % C::STAGES) * C::KV_BYTES;
        for (int i = rloc; i < PG_BK * 8; i += CV_TILE)
          if (!(d.valid >> (i / 8) & 1)) {
#pragma unroll
            for (int b = 0; b < C::DK; ++b) reinterpret_cast<uint4*>(vb + b * PG_BK * 128)[i] = make_uint4(0, 0, 0, 0);
          }
      }
      // row rloc of a K-major 128-byte-swizzled tile: 16-byte chunk c lands at c ^ (row & 7)
#pragma unroll
      for (int ch = 0; ch < 8; ++ch)
        *reinterpret_cast<uint4*>(pdst + ((ch ^ (rloc & 7)) << 4)) =
            make_uint4(pk[4 * ch], pk[4 * ch + 1], pk[4 * ch + 2], pk[4 * ch + 3]);
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive(&p_full[wg]);
      ++n_s;
      if (!(d.flags & TOK_LAST)) continue;

      // ------------- the tile's end: its rows, or their partial slot -------------
      ok = __all_sync(0xffffffffu, mbar_wait(&o_done[wg], (n_s - 1) & 1, p.err) && !*abort_flag);
      if (!ok) break;
      tc_fence_after();
      const bool whole = d.flags & TOK_WHOLE;
      const float inv = lsum == 0.f ? 0.f : 1.f / lsum;
      const int64_t row = live ? paged_out_row(p, d.t0, r, d.h) : 0;
      const int64_t slot = static_cast<int64_t>(blockIdx.x) * 2 + (d.flags & TOK_SLOT1 ? 1 : 0);
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += 16) {
        float v[16];
        tmem_ld16(o_col + c0, v);
        if (!live) continue;
        if (whole) {
          uint4* dst = reinterpret_cast<uint4*>(p.o + row * D + c0);
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] *= inv;
          dst[0] = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                              pack_bf16x2(v[6], v[7]));
          dst[1] = make_uint4(pack_bf16x2(v[8], v[9]), pack_bf16x2(v[10], v[11]), pack_bf16x2(v[12], v[13]),
                              pack_bf16x2(v[14], v[15]));
        } else {
#pragma unroll
          for (int e = 0; e < 16; e += 4)
            *reinterpret_cast<float4*>(p.part + paged_part_at<CV_ROWS, D>(slot, wg * CV_TILE + rloc, c0 + e)) =
                make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
        }
      }
      tc_fence_before();
      mbar_arrive(&o_free[wg]);
      if (live) {
        if (!whole)
          p.part_ml[slot * CV_ROWS + wg * CV_TILE + rloc] = make_float2(mref, lsum);
        else if (p.lse)
          p.lse[row] = lsum == 0.f ? -INFINITY : (mref + log2f(lsum)) * 0.69314718055994531f;
      }
    }
    if (!ok) *abort_flag = 1;
  }
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) paged_poison<CV_ROWS, D>(p, g);
  if (warp == 2) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

}  // namespace dg
