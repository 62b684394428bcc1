// Requests of different lengths over one pool of key/value pages: the block
// tables, slots and positions of a call's new rows, the rows' way into the
// pages, and their attention over them.
//
// Layouts: K and V pools [n_pages][Hkv][page_size][D] bf16 (one head's part of
// a page is contiguous); block table [batch][width] page ids; a slot is
// page * page_size + offset; rows of a call are packed, request b's being
// [cu_rows[b], cu_rows[b + 1]).
#pragma once

#include "common.cuh"

namespace dg {

// Every kernel here may start while the one before it in the stream still
// runs (programmatic dependent launch): it lets the next one start at once,
// sets itself up, and waits for the one before it, all of it, ahead of its
// first access to global memory.  A CTA that leaves early has waited too, so
// the end of a kernel is the end of everything before it.
__device__ __forceinline__ void pdl_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// two floats to bf16, nearest even, lo in the low half
__device__ __forceinline__ uint32_t cvt_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ int64_t min64(int64_t a, int64_t b) { return a < b ? a : b; }
__device__ __forceinline__ int64_t max64(int64_t a, int64_t b) { return a > b ? a : b; }

// ----------------------------------------------------------------------------
// Plan.  With held = ceil(c / page), need = ceil((c + n) / page) for a request
// of cached length c and n new rows (n < 0: its last -n tokens go), the call
// takes max(0, need - held) pages from the head of the ring of free pages and
// puts max(0, held - need) behind its tail, in (request, page) order.  Pages
// taken and pages put are disjoint stretches of the ring, and the counters go
// to another buffer, so no CTA waits for another.
//
// All or nothing: when a length, a row count or the table's width does not
// fit, or the free pages do not suffice, nothing is taken or given back.
//
// Bound by latency (the ids and lengths of 200 requests are 0.2 MB): every CTA
// sums the whole batch's lengths itself (two loads per 256 requests and thread)
// instead of a second launch, then writes its own requests.  2.6 us for one
// request of 256 rows, 4.5 us for 200 requests of 25,000.
// ----------------------------------------------------------------------------
constexpr int PLAN_THREADS = 256;
enum PlanBad : int { PLAN_BAD_LENGTH = 1, PLAN_BAD_WIDTH = 2, PLAN_BAD_ROWS = 4, PLAN_BAD_STATE = 8 };

struct PagedPlanParams {
  const int32_t* cached;
  const int32_t* fresh;        // new rows of each request
  int32_t* table;              // [batch][width], row stride table_stride
  int64_t table_stride;
  int32_t* ring;               // [n_pages] free page ids
  const int32_t* state;        // {head, n_free}
  int32_t* cu_rows;            // [batch + 1]
  int32_t* kv_lens;            // [batch]
  int32_t* positions;          // [row_cap]
  int32_t* slots;              // [row_cap]
  int32_t* state_out;          // {head, n_free, missing pages, PlanBad bits}
  int batch, width, n_pages, page_shift, row_cap;
};

struct PlanRequest {
  int c, n, held, need;
  int bad;
};

__device__ __forceinline__ PlanRequest plan_request(const PagedPlanParams& p, int b) {
  PlanRequest r;
  r.c = p.cached[b];
  r.n = p.fresh[b];
  const int64_t total = static_cast<int64_t>(r.c) + r.n;
  const int64_t up = (int64_t(1) << p.page_shift) - 1;
  r.bad = (r.c < 0 || total < 0 || total > INT32_MAX) ? PLAN_BAD_LENGTH : 0;
  const int64_t held = r.bad ? 0 : (r.c + up) >> p.page_shift;
  const int64_t need = r.bad ? 0 : (total + up) >> p.page_shift;
  if (held > p.width || need > p.width) r.bad |= PLAN_BAD_WIDTH;
  r.held = static_cast<int>(held);
  r.need = static_cast<int>(need);
  return r;
}

__global__ void __launch_bounds__(PLAN_THREADS) paged_plan_kernel(const __grid_constant__ PagedPlanParams p) {
  __shared__ long long red[7][PLAN_THREADS / 32];
  const int b0 = static_cast<int>(static_cast<int64_t>(blockIdx.x) * p.batch / gridDim.x);
  const int b1 = static_cast<int>(static_cast<int64_t>(blockIdx.x + 1) * p.batch / gridDim.x);
  pdl_launch_dependents();
  pdl_wait();
  DG_TIMELINE_SCOPE(TLK_PAGED_PLAN);
  // sums before b0 (rows, grow, back), over the batch (rows, grow, back), bad bits
  long long v[7] = {0, 0, 0, 0, 0, 0, 0};
  for (int b = threadIdx.x; b < p.batch; b += PLAN_THREADS) {
    const PlanRequest r = plan_request(p, b);
    const long long rows = max(r.n, 0), grow = max(r.need - r.held, 0), back = max(r.held - r.need, 0);
    if (b < b0) {
      v[0] += rows;
      v[1] += grow;
      v[2] += back;
    }
    v[3] += rows;
    v[4] += grow;
    v[5] += back;
    v[6] |= r.bad;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
#pragma unroll
    for (int i = 0; i < 6; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    v[6] |= __shfl_xor_sync(0xffffffffu, v[6], o);
  }
  if ((threadIdx.x & 31) == 0)
    for (int i = 0; i < 7; ++i) red[i][threadIdx.x >> 5] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 7; ++i) {
    long long s = 0;
    for (int w = 0; w < PLAN_THREADS / 32; ++w) s = i < 6 ? s + red[i][w] : (s | red[i][w]);
    v[i] = s;
  }
  const int64_t head = p.state[0], n_free = p.state[1];
  const int64_t rows_all = v[3], grow_all = v[4], back_all = v[5];
  int bad = static_cast<int>(v[6]);
  if (rows_all > p.row_cap) bad |= PLAN_BAD_ROWS;
  if (head < 0 || head >= p.n_pages || n_free < 0 || n_free + back_all > p.n_pages) bad |= PLAN_BAD_STATE;
  const bool fits = bad == 0 && grow_all <= n_free;
  const int shift = p.page_shift, mask = (1 << shift) - 1;

  int64_t row0 = v[0], grow0 = v[1], back0 = v[2];
  const bool first_strip = blockIdx.y == 0;
  for (int b = b0; b < b1; ++b) {
    const PlanRequest r = plan_request(p, b);
    const int rows = max(r.n, 0);
    int32_t* tab = p.table + b * p.table_stride;
    if (first_strip && threadIdx.x == 0) {
      p.cu_rows[b] = static_cast<int32_t>(min64(row0, INT32_MAX));
      p.kv_lens[b] = fits ? r.c + r.n : r.c;
    }
    const int64_t take = head + grow0, put = head + n_free + back0;
    if (fits && first_strip) {
      for (int q = r.held + threadIdx.x; q < r.need; q += PLAN_THREADS)
        tab[q] = p.ring[(take + q - r.held) % p.n_pages];
      for (int q = r.need + threadIdx.x; q < r.held; q += PLAN_THREADS)
        p.ring[(put + q - r.need) % p.n_pages] = tab[q];
    }
    const int64_t live = min64(rows, p.row_cap - row0);
    for (int64_t i = blockIdx.y * PLAN_THREADS + threadIdx.x; i < live; i += gridDim.y * PLAN_THREADS) {
      const int64_t pos = max(r.c, 0) + i;
      int32_t slot = -1;
      if (fits) {
        const int q = static_cast<int>(pos >> shift);
        const int64_t page = q < r.held ? tab[q] : p.ring[(take + q - r.held) % p.n_pages];
        if (page >= 0 && page < p.n_pages) slot = static_cast<int32_t>((page << shift) + (pos & mask));
      }
      p.positions[row0 + i] = static_cast<int32_t>(min64(pos, INT32_MAX));
      p.slots[row0 + i] = slot;
    }
    row0 += rows;
    grow0 += max(r.need - r.held, 0);
    back0 += max(r.held - r.need, 0);
  }
  if (b1 == p.batch && first_strip && threadIdx.x == 0) {
    p.cu_rows[p.batch] = static_cast<int32_t>(min64(rows_all, INT32_MAX));
    p.state_out[0] = fits ? static_cast<int32_t>((head + grow_all) % p.n_pages) : static_cast<int32_t>(head);
    p.state_out[1] = static_cast<int32_t>(fits ? n_free - grow_all + back_all : n_free);
    p.state_out[2] = static_cast<int32_t>(min64(max64(grow_all - n_free, 0), INT32_MAX));
    p.state_out[3] = bad;
  }
}

// ----------------------------------------------------------------------------
// Append.  Rotates the pairs (j, j + D/2) of q and k by the angles of the
// row's position, x_j' = x_j cos - x_{j+D/2} sin, x_{j+D/2}' = x_{j+D/2} cos +
// x_j sin, in fp32, rounds once to bf16, and writes q packed, k and v to the
// row's slot.
//
// Bound by HBM: 2 x (Hq + 2 Hkv) x D x 2 bytes a row.  A thread takes eight
// pairs (two 16-byte loads) of APPEND_HEADS heads, so the eight (cos, sin) of a
// chunk are loaded once for them and eight loads are in flight per thread.
// 16,000 rows of 16/8 heads of 176: 56.2 us, 6.4 TB/s (0.99 of the copy peak);
// 62 us with 256 threads, 63 with two heads a thread, 65 with eight.
// ----------------------------------------------------------------------------
constexpr int APPEND_THREADS = 128;
constexpr int APPEND_HEADS = 4;

struct PagedAppendParams {
  const uint16_t* qkv;         // [rows][(Hq + 2 Hkv) D], row stride qkv_stride
  int64_t qkv_stride;
  const float* part;           // or the split-K sums of the projection [splits][rows][(Hq + 2 Hkv) D], added in order
  int splits;
  const int32_t* positions;
  const int32_t* slots;
  const float4* rope;          // [n_positions][D/2] (cos, sin)
  uint16_t* k;
  uint16_t* v;
  uint16_t* q;                 // [rows][Hq][D]
  int64_t n_slots;             // n_pages * page_size
  int rows, n_positions, Hq, Hkv, page_shift;
};

__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(cvt_bf16x2(f[0], f[1]), cvt_bf16x2(f[2], f[3]), cvt_bf16x2(f[4], f[5]),
                    cvt_bf16x2(f[6], f[7]));
}

// eight columns of a row as fp32: split sums added in order, or bf16 values
template <bool SPLITS>
struct AppendIn {
  float f[8];
  __device__ __forceinline__ void load(const PagedAppendParams& p, int64_t row, int64_t width, int64_t col) {
    const float* src = p.part + row * width + col;
    float4 a = *reinterpret_cast<const float4*>(src), b = *reinterpret_cast<const float4*>(src + 4);
    for (int s = 1; s < p.splits; ++s) {
      src += p.rows * width;
      const float4 x = *reinterpret_cast<const float4*>(src), y = *reinterpret_cast<const float4*>(src + 4);
      a = make_float4(a.x + x.x, a.y + x.y, a.z + x.z, a.w + x.w);
      b = make_float4(b.x + y.x, b.y + y.y, b.z + y.z, b.w + y.w);
    }
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = f[e];
  }
  __device__ __forceinline__ uint4 bits() const { return pack8(f); }
};
template <>
struct AppendIn<false> {
  uint4 u;
  __device__ __forceinline__ void load(const PagedAppendParams& p, int64_t row, int64_t, int64_t col) {
    u = *reinterpret_cast<const uint4*>(p.qkv + row * p.qkv_stride + col);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const { unpack8(u, v); }
  __device__ __forceinline__ uint4 bits() const { return u; }
};

template <int D, bool SPLITS>
__global__ void __launch_bounds__(APPEND_THREADS) paged_append_kernel(const __grid_constant__ PagedAppendParams p) {
  constexpr int HALF = D / 2, C = HALF / 8;  // chunks of eight pairs in a head
  static_assert(HALF % 8 == 0, "16-byte halves");
  const int heads = p.Hq + 2 * p.Hkv, groups = (heads + APPEND_HEADS - 1) / APPEND_HEADS;
  const int64_t it = static_cast<int64_t>(blockIdx.x) * APPEND_THREADS + threadIdx.x;
  pdl_launch_dependents();
  pdl_wait();
  DG_TIMELINE_SCOPE(TLK_PAGED_APPEND);
  if (it >= static_cast<int64_t>(p.rows) * groups * C) return;
  const int c = static_cast<int>(it % C);
  const int h0 = static_cast<int>(it / C % groups) * APPEND_HEADS;
  const int64_t row = it / C / groups;
  const int pos = p.positions[row], slot = p.slots[row];
  const bool known = pos >= 0 && pos < p.n_positions;
  const bool kept = known && slot >= 0 && slot < p.n_slots;
  AppendIn<SPLITS> lo[APPEND_HEADS], hi[APPEND_HEADS];
#pragma unroll
  for (int i = 0; i < APPEND_HEADS; ++i)
    if (h0 + i < heads) {
      lo[i].load(p, row, heads * D, (h0 + i) * D + c * 8);
      hi[i].load(p, row, heads * D, (h0 + i) * D + c * 8 + HALF);
    }
  float cs[8], sn[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // a position the table does not hold has no angle: its q row comes back NaN
    const float4 t = known ? p.rope[(static_cast<int64_t>(pos) * HALF + c * 8) / 2 + i] : make_float4(NAN, NAN, NAN, NAN);
    cs[2 * i] = t.x;
    sn[2 * i] = t.y;
    cs[2 * i + 1] = t.z;
    sn[2 * i + 1] = t.w;
  }
  const int page = slot >> p.page_shift, off = slot & ((1 << p.page_shift) - 1);
#pragma unroll
  for (int i = 0; i < APPEND_HEADS; ++i) {
    const int h = h0 + i;
    if (h >= heads) break;
    uint4 out_lo, out_hi;
    if (h < p.Hq + p.Hkv) {
      float a[8], b[8], x[8], y[8];
      lo[i].get(a);
      hi[i].get(b);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] = a[e] * cs[e] - b[e] * sn[e];
        y[e] = b[e] * cs[e] + a[e] * sn[e];
      }
      out_lo = pack8(x);
      out_hi = pack8(y);
    } else {
      out_lo = lo[i].bits();
      out_hi = hi[i].bits();
    }
    uint16_t* dst;
    if (h < p.Hq) {
      dst = p.q + (row * p.Hq + h) * D;
    } else {
      if (!kept) continue;
      const int g = h < p.Hq + p.Hkv ? h - p.Hq : h - p.Hq - p.Hkv;
      dst = (h < p.Hq + p.Hkv ? p.k : p.v) +
            (((static_cast<int64_t>(page) * p.Hkv + g) << p.page_shift) + off) * D;
    }
    *reinterpret_cast<uint4*>(dst + c * 8) = out_lo;
    *reinterpret_cast<uint4*>(dst + c * 8 + HALF) = out_hi;
  }
}

}  // namespace dg
