// Filling an 8-bit paged key-value cache and taking its values out again (sage_paged_append_q8, sage_paged_read_q8).
//
// The scale of a block follows its tokens: the largest magnitude among them decides it (needed_scale). A token that joins
// a block whose scale is too small raises the scale to what it needs, and the codes of the block's earlier tokens are
// rounded again to the new one: for E4M3 that moves an exponent and is exact but for subnormals; for int8 it adds at most
// half a step for each time a block's scale grows, which for tokens of one distribution is a few times in a block.
//
// DRAM bounds both for prompts: 41K tokens of 8 heads, head_dim 128, K and V (243 MB, 36 us at a copy's rate): append 42 to 50 us by
// the size of the blocks (43 at 64 tokens), read 46 to 49.
#include <cmath>

#include "../../include/sageattn.h"
#include "launch.h"
#include "paged_q8.cuh"

namespace sage {

int make_q8_view(const sage_q8_cache* c, int batch, int heads_kv, int head_dim, int layout, Q8View* view, int* align) {
  if (!c) return SAGE_ERR_INVALID_ARG;
  if (head_dim < 1 || head_dim > 128) return SAGE_ERR_HEAD_DIM;
  if ((c->k_type != SAGE_S8 && c->k_type != SAGE_E4M3) || (c->v_type != SAGE_S8 && c->v_type != SAGE_E4M3))
    return SAGE_ERR_DTYPE;
  if (layout != SAGE_HND && layout != SAGE_NHD) return SAGE_ERR_INVALID_ARG;
  if (batch < 0 || heads_kv < 1 || heads_kv > 65535 || c->num_pages < 0 || c->page_size < 1 || c->max_pages < 0 ||
      c->block < 1 || c->page_size % c->block || (int64_t)c->max_pages * c->page_size > kMostSlots)
    return SAGE_ERR_INVALID_ARG;
  if (batch > 0) {
    auto off = [](const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; };
    if ((!c->page_table && c->max_pages > 0) || !c->seq_lens || off(c->page_table, 4) || off(c->seq_lens, 4) ||
        off(c->k_scales, 4) || off(c->v_scales, 4) || c->table_stride < 0)
      return SAGE_ERR_INVALID_ARG;
    if (c->num_pages > 0 && (!c->k || !c->v || !c->k_scales || !c->v_scales)) return SAGE_ERR_INVALID_ARG;
    for (int i = 0; i < 3; ++i)
      if (c->k_stride[i] < 0 || c->v_stride[i] < 0) return SAGE_ERR_STRIDE;
  }
  Q8View q{};
  PagedView& v = q.c;
  v.batch = batch; v.hkv = heads_kv; v.d = head_dim;
  v.page_size = c->page_size; v.num_pages = c->num_pages; v.max_pages = c->max_pages;
  const int hi = layout == SAGE_HND ? 1 : 2, ti = layout == SAGE_HND ? 2 : 1;
  v.k = c->k; v.k_sp = c->k_stride[0]; v.k_sh = c->k_stride[hi]; v.k_st = c->k_stride[ti];
  v.v = c->v; v.v_sp = c->v_stride[0]; v.v_sh = c->v_stride[hi]; v.v_st = c->v_stride[ti];
  v.table = c->page_table; v.table_stride = c->table_stride; v.lens = c->seq_lens;
  q.ks = c->k_scales; q.vs = c->v_scales;
  q.block = c->block; q.blocks = c->page_size / c->block;
  q.k_type = c->k_type; q.v_type = c->v_type;
  int w = 16;
  auto fits = [&](uint64_t x) { while (x % w) w /= 2; };
  fits(reinterpret_cast<uintptr_t>(c->k));
  fits(reinterpret_cast<uintptr_t>(c->v));
  fits(head_dim);
  if (c->num_pages > 1) { fits(v.k_sp); fits(v.v_sp); }
  if (heads_kv > 1) { fits(v.k_sh); fits(v.v_sh); }
  if (c->page_size > 1) { fits(v.k_st); fits(v.v_st); }
  *view = q;
  *align = w;
  return SAGE_OK;
}

namespace {

// The sequence of row t, the last b with cu[b] <= t (batch: behind the last one): a warp looks at 32 places at a time, so
// 1024 sequences take two dependent loads where a bisection takes ten.
__device__ __forceinline__ int sequence_of(const int* cu, int batch, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = batch + 1;  // among lo .. lo + n - 1
  while (n > 1) {
    const int step = (n + 31) / 32, at = lane * step;
    const bool le = at < n && __ldg(&cu[lo + at]) <= t;
    const unsigned set = __ballot_sync(0xffffffffu, le);
    const int last = set ? 31 - __clz(set) : 0;
    lo += last * step;
    n = min(step, n - last * step);
  }
  return lo;
}

// ------------------------------------------------------------------------------------- append
struct AppendArgs {
  Q8View q;
  const void* x[2]; int64_t x_st[2], x_sh[2];  // k, v: element strides of token and head
  const int* cu;        // [batch + 1] or null: one token per sequence
  int tokens, chunk;    // rows that a CTA looks after
  int shares;           // CTAs that share a chunk's heads
  int window;           // slots that are written together: whole blocks of one page
  int in_run, out_run;  // channels of a row's loads and of the codes' stores: 8, 4 or 1
  int lanes;            // lanes of a row, 8 channels each: 4, 8 or 16
  int block_shift;      // log2 of the block, or -1
  int* err;             // or null
};

// A window takes one of these forms. kOne: one block, by a warp. kMany: several small blocks, by a warp, whose rows' largest
// magnitudes and scales meet in shared memory. kTwo, kFour, kEight: one block, by a CTA of so many warps: as many as hold
// its rows in registers (us for 41K tokens of 8 heads of head_dim 128, K and V: blocks of 32 by two warps 42, by four 59; of 128 by
// eight 48, by four, which read half of the rows twice, 73).
enum { kOne, kMany, kTwo, kFour, kEight };
__host__ __device__ constexpr int warps_of(int form) { return form == kTwo ? 2 : form == kEight ? 8 : 4; }
__host__ __device__ constexpr bool by_cta(int form) { return form >= kTwo; }
constexpr int kManyRows = 32;  // of a window of several blocks
constexpr int kKept = 8;  // rows of a lane that stay in registers between the two walks over them

// New rows of a window: the first one's token, how many; the page, slot and block of the first; earlier tokens of its block.
struct Window {
  int64_t row0;
  int rows, page, slot0, block0, held;
};

// Eight channels of a row from ch on, which is one of it; zeros past the last. FULL: all rows and codes allow runs of eight.
template <typename T, bool FULL>
__device__ __forceinline__ uint4 load_run(const AppendArgs& a, const T* row, int ch) {
  if (FULL || a.in_run == 8) return __ldg(reinterpret_cast<const uint4*>(row + ch));
  if (a.in_run == 4) {
    const uint2 lo = __ldg(reinterpret_cast<const uint2*>(row + ch));
    const uint2 hi = ch + 4 < a.q.c.d ? __ldg(reinterpret_cast<const uint2*>(row + ch + 4)) : make_uint2(0, 0);
    return make_uint4(lo.x, lo.y, hi.x, hi.y);
  }
  return load8_raw<T>(row, ch, a.q.c.d, 0);
}

// Rows of one unit (a head's K or V) for this lane: the first kKept of them.
template <typename T, int FORM, bool FULL>
__device__ __forceinline__ void fetch_rows(const AppendArgs& a, const Window& w, int unit, uint4 (&kept)[kKept]) {
  const int lane = threadIdx.x & 31, ch = (lane & (a.lanes - 1)) * 8, per = 32 / a.lanes;
  const int kv = unit >= a.q.c.hkv, h = unit - kv * a.q.c.hkv, step = by_cta(FORM) ? per * warps_of(FORM) : per;
  const int first = (by_cta(FORM) ? (threadIdx.x >> 5) * per : 0) + lane / a.lanes;
  const T* x = static_cast<const T*>(a.x[kv]) + (w.row0 + first) * a.x_st[kv] + h * a.x_sh[kv];
  const int64_t jump = step * a.x_st[kv];
#pragma unroll
  for (int i = 0; i < kKept; ++i) {
    kept[i] = make_uint4(0, 0, 0, 0);
    if (ch < a.q.c.d && first + i * step < w.rows) kept[i] = load_run<T, FULL>(a, x, ch);
    x += jump;
  }
}

// Largest magnitude of a run of eight, as bit patterns, whose order is that of the magnitudes: a pair of them.
__device__ __forceinline__ uint32_t largest2(const uint4& raw, uint32_t m) {
  constexpr uint32_t kAbs = 0x7fff7fffu;
  m = __vmaxu2(m, raw.x & kAbs);
  m = __vmaxu2(m, raw.y & kAbs);
  m = __vmaxu2(m, raw.z & kAbs);
  return __vmaxu2(m, raw.w & kAbs);
}
template <typename T>
__device__ __forceinline__ float pattern(uint32_t pair) {
  const uint16_t m = (uint16_t)max(pair & 0xffffu, pair >> 16);
  return to_f32<T>(*reinterpret_cast<const T*>(&m));
}
template <typename T>
__device__ __forceinline__ void widen8(const uint4& raw, float (&f)[8]) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (std::is_same<T, __half>::value) {
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = v.x;
      f[2 * i + 1] = v.y;
    } else {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

// The largest magnitude of each block, its scale, the codes.
template <typename T, int TYPE, int FORM, bool FULL>
__device__ __forceinline__ void store_window(const AppendArgs& a, const Window& w, int unit, uint4 (&kept)[kKept], float* s_most) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const PagedView& c = a.q.c;
  const int kv = unit >= a.q.c.hkv, h = unit - kv * a.q.c.hkv;
  const int ch = (lane & (a.lanes - 1)) * 8, per = 32 / a.lanes, step = by_cta(FORM) ? per * warps_of(FORM) : per;
  const int first = (by_cta(FORM) ? warp * per : 0) + lane / a.lanes;
  const bool on = ch < c.d;
  const T* x = static_cast<const T*>(a.x[kv]) + w.row0 * a.x_st[kv] + h * a.x_sh[kv];
  const int64_t xs = a.x_st[kv], cs = kv ? c.v_st : c.k_st;
  uint8_t* base = static_cast<uint8_t*>(kv ? c.v : c.k) + w.page * (kv ? c.v_sp : c.k_sp) + h * (kv ? c.v_sh : c.k_sh) + ch;
  float* const scales = (kv ? a.q.vs : a.q.ks) + ((int64_t)w.page * c.hkv + h) * a.q.blocks;
  const int block0 = w.block0;
  const float was = w.held ? scales[block0] : 0.f;
  auto put = [&](uint8_t* d, const uint2& code) {
    if (FULL || a.out_run == 8) {
      *reinterpret_cast<uint2*>(d) = code;
    } else if (a.out_run == 4) {
      *reinterpret_cast<uint32_t*>(d) = code.x;
      if (ch + 4 < c.d) *reinterpret_cast<uint32_t*>(d + 4) = code.y;
    } else {
      const uint8_t* b = reinterpret_cast<const uint8_t*>(&code);
      for (int e = 0; e < 8; ++e)
        if (ch + e < c.d) d[e] = b[e];
    }
  };
  uint8_t* to = base + (int64_t)(w.slot0 + first) * cs;  // this lane's next row
  const int64_t hop = step * cs;
  auto write = [&](const uint4& raw, float inv) {
    float u[8];
    widen8<T>(raw, u);
#pragma unroll
    for (int e = 0; e < 8; ++e) u[e] = __fmul_rn(u[e], inv);
    put(to, to_codes<TYPE>(u));
  };
  // the earlier codes of the first block, where its scale has grown
  auto again = [&](float scale) {
    if (!w.held || !(scale > was)) return;
    const float f = __fdiv_rn(was, scale);
    for (int r = first; r < w.held; r += step) {
      if (!on) break;
      uint8_t* s = base + (int64_t)(w.slot0 - w.held + r) * cs;
      alignas(8) uint8_t code[8];
      if (FULL || a.out_run == 8) {
        *reinterpret_cast<uint2*>(code) = *reinterpret_cast<const uint2*>(s);
      } else {
        for (int e = 0; e < 8; ++e) code[e] = ch + e < c.d ? s[e] : 0;
      }
      float u[8];
      from_codes<TYPE>(reinterpret_cast<const uint32_t*>(code)[0], u[0], u[1], u[2], u[3]);
      from_codes<TYPE>(reinterpret_cast<const uint32_t*>(code)[1], u[4], u[5], u[6], u[7]);
#pragma unroll
      for (int e = 0; e < 8; ++e) u[e] = __fmul_rn(u[e], f);
      put(s, to_codes<TYPE>(u, true));
    }
  };
  if constexpr (FORM == kMany) {
    // a row's largest magnitude, then each block's over its rows, by a lane each
    float* const s_scale = s_most + kManyRows;  // [2][kManyRows]: scales, their reciprocals
    // (the lanes of a row halve the rows twice while they exchange, two rows in a register)
    const int far = a.lanes / 2, near = a.lanes / 4;
    const bool up = lane & far, up2 = lane & near;
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t x = largest2(kept[2 * i], 0), y = largest2(kept[2 * i + 1], 0);
      q[i] = __vmaxu2(__byte_perm(x, y, 0x5410), __byte_perm(x, y, 0x7632));
    }
    const uint32_t x0 = __vmaxu2(up ? q[2] : q[0], __shfl_xor_sync(0xffffffffu, up ? q[0] : q[2], far));
    const uint32_t x1 = __vmaxu2(up ? q[3] : q[1], __shfl_xor_sync(0xffffffffu, up ? q[1] : q[3], far));
    uint32_t m2 = __vmaxu2(up2 ? x1 : x0, __shfl_xor_sync(0xffffffffu, up2 ? x0 : x1, near));
    for (int o = near / 2; o > 0; o >>= 1) m2 = __vmaxu2(m2, __shfl_xor_sync(0xffffffffu, m2, o));
    if ((lane & (near - 1)) == 0) {
      const int row = first + ((up ? 4 : 0) + (up2 ? 2 : 0)) * step;
      if (row < w.rows) s_most[row] = pattern<T>(m2 & 0xffffu);
      if (row + step < w.rows) s_most[row + step] = pattern<T>(m2 >> 16);
    }
    __syncwarp();  // (also: every lane has read the old scale)
    if (lane * a.q.block < w.held + w.rows) {
      float m = 0.f;
      const int end = min(w.rows, (lane + 1) * a.q.block - w.held);
      for (int r = max(0, lane * a.q.block - w.held); r < end; ++r) m = fmaxf(m, s_most[r]);
      const float scale = fmaxf(lane == 0 ? was : 0.f, needed_scale<TYPE>(m));
      s_scale[lane] = scale;
      s_scale[kManyRows + lane] = __frcp_rn(scale);
      scales[block0 + lane] = scale;
    }
    __syncwarp();
    if (w.held) again(s_scale[0]);
#pragma unroll
    for (int i = 0; i < kKept; ++i) {
      const int r = first + i * step, block = a.block_shift >= 0 ? (w.held + r) >> a.block_shift : (w.held + r) / a.q.block;
      if (on && r < w.rows) write(kept[i], s_scale[kManyRows + block]);
      to += hop;
    }
    __syncwarp();  // (the next unit writes there)
  } else {
    uint32_t pair = 0;
#pragma unroll
    for (int i = 0; i < kKept; ++i) pair = largest2(kept[i], pair);
    for (int r = first + kKept * step; r < w.rows; r += step)
      if (on) pair = largest2(load_run<T, FULL>(a, x + r * xs, ch), pair);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) pair = __vmaxu2(pair, __shfl_xor_sync(0xffffffffu, pair, o));
    float most = pattern<T>(pair);
    if (by_cta(FORM)) {
      __syncthreads();  // (also: every thread has read the old scale)
      if (lane == 0) s_most[warp] = most;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < warps_of(FORM); ++i) most = fmaxf(most, s_most[i]);
    }
    const float scale = fmaxf(was, needed_scale<TYPE>(most)), inv = __frcp_rn(scale);
    __syncwarp();  // (every lane has read the old scale)
    if (by_cta(FORM) ? threadIdx.x == 0 : lane == 0) scales[block0] = scale;
    again(scale);
#pragma unroll
    for (int i = 0; i < kKept; ++i) {
      if (on && first + i * step < w.rows) write(kept[i], inv);
      to += hop;
    }
    for (int r = first + kKept * step; r < w.rows; r += step) {
      if (on) write(load_run<T, FULL>(a, x + r * xs, ch), inv);
      to += hop;
    }
  }
}

// CTA (x, y) of line x * shares + y: the windows whose first new token lies in rows [x chunk, (x + 1) chunk), for the y-th
// share of the heads' K and V (kTwo to kEight: by the whole CTA, otherwise by a warp each). DRAM bounds it for prompts, which many
// resident warps keep busy: fetching the next head's rows while one is scaled took twice the registers and was slower. At 72
// registers kOne spills 20 to 36 bytes and kMany 4.
template <typename T, int FORM, bool FULL>
__global__ void __launch_bounds__(32 * warps_of(FORM), 28 / warps_of(FORM)) append_q8_kernel(const AppendArgs a) {
  __shared__ float s_most[4][FORM == kMany ? 3 * kManyRows : 8];
  const PagedView& c = a.q.c;
  const int warp = threadIdx.x >> 5, units = 2 * c.hkv;
  const int share = blockIdx.x % a.shares;  // (CTAs of one window run side by side: they read the same token rows)
  const int64_t place = blockIdx.x / a.shares;
  const int unit0 = by_cta(FORM) ? share : share * 4 + warp, unit_step = by_cta(FORM) ? a.shares : a.shares * 4;
  pdl_wait();
  pdl_trigger();
  if (unit0 >= units) return;  // (a whole warp, or no thread of the CTA)
  const bool tells = a.err && unit0 == 0 && (threadIdx.x & 31) == 0 && (!by_cta(FORM) || threadIdx.x == 0);
  const int64_t t_end = min((int64_t)a.tokens, (place + 1) * a.chunk);
  int64_t t = place * a.chunk;
  int b = a.cu ? sequence_of(a.cu, c.batch, (int)t) : (int)t;
  while (t < t_end) {
    int64_t first = t, end = t + 1;
    if (a.cu) {
      first = __ldg(&a.cu[b]);
      if (tells && t == 0 && first != 0) record_error(a.err, kDevSeqlens);
      if (b >= c.batch) return;              // behind the last sequence
      if (first > t) { t = first; continue; }  // before the first: rows that are left out
      end = min((int64_t)__ldg(&a.cu[b + 1]), (int64_t)a.tokens);
      if (end <= t) { ++b; continue; }       // a sequence without tokens (b grows: at most batch of them)
    }
    const int len = __ldg(&c.lens[b]);
    const int64_t room = (int64_t)c.max_pages * c.page_size;
    const int64_t slot = (int64_t)len + t - first;
    int64_t next = end;                      // (without a place: the rest of this sequence)
    if (len < 0 || slot >= room) {
      if (tells) record_error(a.err, kDevSeqlens);
    } else {
      const int i = (int)(slot / c.page_size), s0 = (int)(slot - (int64_t)i * c.page_size), in = s0 % a.window;
      next = min(end, t + min(a.window - in, c.page_size - s0));
      if (t == first || in == 0) {           // the first new token of its window
        const int page = __ldg(&c.table[b * c.table_stride + i]);
        if (page < 0 || page >= c.num_pages) {
          if (tells) record_error(a.err, kDevPage);
        } else {
          const int block0 = s0 / a.q.block;
          const Window w{t, (int)(next - t), page, s0, block0, s0 - block0 * a.q.block};
#pragma unroll 1
          for (int u = unit0; u < units; u += unit_step) {
            uint4 kept[kKept];
            fetch_rows<T, FORM, FULL>(a, w, u, kept);
            if ((u >= c.hkv ? a.q.v_type : a.q.k_type) == SAGE_S8) store_window<T, SAGE_S8, FORM, FULL>(a, w, u, kept, s_most[by_cta(FORM) ? 0 : warp]);
            else store_window<T, SAGE_E4M3, FORM, FULL>(a, w, u, kept, s_most[by_cta(FORM) ? 0 : warp]);
          }
        }
      }
    }
    t = next;
    if (t >= end) {
      if (a.cu) ++b;
      else b = (int)t;
    }
  }
}

// --------------------------------------------------------------------------------------- read
struct ReadArgs {
  Q8View q;
  void* y[2]; int64_t y_st[2], y_sh[2];
  const int* cu; const int* starts;  // starts: first slot of each sequence, or null (0)
  int tokens, rows;  // rows of a warp: up to 32
  int* err;
};

template <typename T>
__device__ __forceinline__ uint32_t narrow2(float lo, float hi) {
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
// Four codes times their scale, in 16 bits.
template <typename T, int TYPE>
__device__ __forceinline__ uint2 values4(uint32_t codes, float scale) {
  float f0, f1, f2, f3;
  from_codes<TYPE>(codes, f0, f1, f2, f3);
  mul2(f0, f1, f0, f1, scale, scale);
  mul2(f2, f3, f2, f3, scale, scale);
  return make_uint2(narrow2<T>(f0, f1), narrow2<T>(f2, f3));
}

// V codes at p as channels at y, or zeros.
template <typename T, int V, int TYPE>
struct CodeRun {
  uint32_t raw[V == 8 ? 2 : 1];
  float scale;
  __device__ __forceinline__ void load(const uint8_t* p, const float* s, bool in) {
    scale = 0.f;
#pragma unroll
    for (uint32_t& w : raw) w = 0;
    if (!in) return;
    scale = __ldg(s);
    if constexpr (V == 8) {
      const uint2 w = __ldg(reinterpret_cast<const uint2*>(p));
      raw[0] = w.x; raw[1] = w.y;
    } else if constexpr (V == 4) {
      raw[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
    } else {
      raw[0] = *p;
    }
  }
  __device__ __forceinline__ void store(T* y) const {
    const uint2 lo = values4<T, TYPE>(raw[0], scale);
    if constexpr (V == 8) {
      const uint2 hi = values4<T, TYPE>(raw[1], scale);
      *reinterpret_cast<uint4*>(y) = make_uint4(lo.x, lo.y, hi.x, hi.y);
    } else if constexpr (V == 4) {
      *reinterpret_cast<uint2*>(y) = lo;
    } else {
      *reinterpret_cast<uint16_t*>(y) = (uint16_t)lo.x;
    }
  }
};

// Rows t0 .. of K or V: lane j knows where row j's codes and first scale lie (no row: -1).
template <typename T, int V, int TYPE>
__device__ __forceinline__ void copy_rows(const ReadArgs& a, int kv, int64_t t0, int n_rows, long long code_at, long long scale_at) {
  const PagedView& c = a.q.c;
  const int lane = threadIdx.x & 31;
  const int64_t sh = kv ? c.v_sh : c.k_sh, ys = a.y_st[kv];
  const uint8_t* codes = static_cast<const uint8_t*>(kv ? c.v : c.k);
  const float* scales = kv ? a.q.vs : a.q.ks;
  T* const y = static_cast<T*>(a.y[kv]) + t0 * ys;
  const int runs = (c.d + V - 1) / V, n = c.hkv * runs;
  CodeRun<T, V, TYPE> run[2];
  if (n <= 32) {
    // short rows: the lanes take the runs of several, two each
    const int side = 32 / n, g = lane / n, x = lane - g * n, h = x / runs, ch = (x - h * runs) * V;
    const uint8_t* src = codes + h * sh + ch;
    const float* sc = scales + (int64_t)h * a.q.blocks;
    T* const dst = y + h * a.y_sh[kv] + ch;
#pragma unroll 1
    for (int j0 = 0; j0 < n_rows; j0 += 2 * side) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int j = j0 + u * side + g;
        const long long at = __shfl_sync(0xffffffffu, code_at, j & 31), sat = __shfl_sync(0xffffffffu, scale_at, j & 31);
        run[u].load(src + at, sc + sat, j < n_rows && at >= 0);
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int j = j0 + u * side + g;
        if (g < side && j < n_rows) run[u].store(dst + j * ys);
      }
    }
    return;
  }
  for (int x0 = 0; x0 < n; x0 += 64) {
    // two runs of a row for each lane
    const uint8_t* src[2];
    const float* sc[2];
    T* dst[2];
    bool on[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int x = x0 + 32 * u + lane, h = x / runs, ch = (x - h * runs) * V;
      on[u] = x < n;
      src[u] = codes + h * sh + ch;
      sc[u] = scales + (int64_t)h * a.q.blocks;
      dst[u] = y + h * a.y_sh[kv] + ch;
    }
#pragma unroll 1
    for (int j = 0; j < n_rows; ++j) {
      const long long at = __shfl_sync(0xffffffffu, code_at, j), sat = __shfl_sync(0xffffffffu, scale_at, j);
#pragma unroll
      for (int u = 0; u < 2; ++u) run[u].load(src[u] + at, sc[u] + sat, on[u] && at >= 0);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (on[u]) run[u].store(dst[u]);
        dst[u] += ys;
      }
    }
  }
}

// A warp per `rows` rows of K or of V (blockIdx.y): its lanes find the rows' places side by side, then take V codes each, the same
// channels of row after row. Few registers and many warps, which keep DRAM busy: four rows of two runs in flight in each of half as
// many warps took 68 us where this took 52 (41K tokens of 8 heads, head_dim 128, caches cold).
template <typename T, int V>
__global__ void __launch_bounds__(128, 10) read_q8_kernel(const ReadArgs a) {
  const PagedView& c = a.q.c;
  const int lane = threadIdx.x & 31, kv = blockIdx.y;
  const int64_t t0 = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 5)) * a.rows;
  pdl_wait();
  pdl_trigger();
  if (t0 >= a.tokens) return;
  const int n_rows = (int)min((int64_t)a.rows, a.tokens - t0);
  int page = -1, slot = 0;
  if (lane < n_rows) {
    const int t = (int)t0 + lane;
    int lo = 0, hi = c.batch;  // the last b with cu[b] <= t
    while (lo < hi) {
      const int mid = lo + (hi - lo + 1) / 2;
      if (__ldg(&a.cu[mid]) <= t) lo = mid;
      else hi = mid - 1;
    }
    const int b = lo, first = __ldg(&a.cu[b]);
    if (a.err && t == 0 && kv == 0 && first != 0) record_error(a.err, kDevSeqlens);
    if (b < c.batch && first <= t) {
      const int len = __ldg(&c.lens[b]);
      const int64_t s = (a.starts ? __ldg(&a.starts[b]) : 0) + (int64_t)t - first;
      if (s < 0 || s >= len || s >= (int64_t)c.max_pages * c.page_size) {
        if (a.err && kv == 0) record_error(a.err, kDevSeqlens);
      } else {
        const int i = (int)(s / c.page_size);
        slot = (int)(s - (int64_t)i * c.page_size);
        page = __ldg(&c.table[b * c.table_stride + i]);
        if (page < 0 || page >= c.num_pages) {
          page = -1;
          if (a.err && kv == 0) record_error(a.err, kDevPage);
        }
      }
    }
  }
  // where this lane's row and its first scale lie
  const long long code_at = page >= 0 ? page * (kv ? c.v_sp : c.k_sp) + slot * (kv ? c.v_st : c.k_st) : -1;
  const long long scale_at = page >= 0 ? (long long)page * c.hkv * a.q.blocks + slot / a.q.block : 0;
  if ((kv ? a.q.v_type : a.q.k_type) == SAGE_S8) copy_rows<T, V, SAGE_S8>(a, kv, t0, n_rows, code_at, scale_at);
  else copy_rows<T, V, SAGE_E4M3>(a, kv, t0, n_rows, code_at, scale_at);
}

int check_status_word(const void* workspace, size_t bytes) {
  return workspace && (reinterpret_cast<uintptr_t>(workspace) % 256 || bytes < SAGE_STATUS_BYTES) ? SAGE_ERR_WORKSPACE
                                                                                                 : SAGE_OK;
}
// A packed operand of rows; *run: channels that an access of every row can take, 8, 4 or 1.
int check_rows(const sage_packed* t, int tokens, int heads, int d, bool written, int* run) {
  if (!t->data) return SAGE_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(t->data) % 2 || t->stride_token < 0 || t->stride_head < 0) return SAGE_ERR_STRIDE;
  if (written && ((tokens > 1 && t->stride_token == 0) || (heads > 1 && t->stride_head == 0))) return SAGE_ERR_STRIDE;
  auto fits = [&](int n) {
    return reinterpret_cast<uintptr_t>(t->data) % (2 * n) == 0 && d % n == 0 && (tokens <= 1 || t->stride_token % n == 0) &&
           (heads <= 1 || t->stride_head % n == 0);
  };
  *run = *run == 8 && fits(8) ? 8 : *run >= 4 && fits(4) ? 4 : 1;
  return SAGE_OK;
}

}  // namespace
}  // namespace sage

using namespace sage;

extern "C" {

int sage_paged_append_q8(const sage_packed* k, const sage_packed* v, const sage_q8_cache* cache, const int32_t* cu_seqlens,
                         int batch, int tokens, int heads_kv, int head_dim, int dtype, int tensor_layout, void* workspace,
                         size_t workspace_bytes, void* stream) {
  if (!k || !v) return SAGE_ERR_INVALID_ARG;
  AppendArgs a{};
  int align = 1;
  int s = make_q8_view(cache, batch, heads_kv, head_dim, tensor_layout, &a.q, &align);
  if (s != SAGE_OK) return s;
  if (dtype != SAGE_F16 && dtype != SAGE_BF16) return SAGE_ERR_DTYPE;
  if (tokens < 0 || (!cu_seqlens && tokens != batch) || reinterpret_cast<uintptr_t>(cu_seqlens) % 4) return SAGE_ERR_INVALID_ARG;
  if (check_status_word(workspace, workspace_bytes) != SAGE_OK) return SAGE_ERR_WORKSPACE;
  if (batch == 0 || tokens == 0) return empty_call(workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
  int run = 8;
  const sage_packed* t[2] = {k, v};
  for (int i = 0; i < 2; ++i) {
    s = check_rows(t[i], tokens, heads_kv, head_dim, false, &run);
    if (s != SAGE_OK) return s;
    a.x[i] = t[i]->data;
    a.x_st[i] = t[i]->stride_token;
    a.x_sh[i] = t[i]->stride_head;
  }
  if (!sage_device_supported()) return SAGE_ERR_DEVICE;
  a.cu = cu_seqlens;
  a.tokens = tokens;
  a.in_run = run;
  a.out_run = align >= 8 ? 8 : align >= 4 ? 4 : 1;  // (and head_dim a multiple of it)
  a.lanes = head_dim <= 32 ? 4 : head_dim <= 64 ? 8 : 16;
  a.err = static_cast<int*>(workspace);
  // a window: a block, or as many small ones as a warp's registers hold rows of
  const int hold = kKept * (32 / a.lanes), block = a.q.block;
  a.block_shift = -1;
  for (int i = 0; i < 31; ++i)
    if (block == 1 << i) a.block_shift = i;
  const int many = hold < kManyRows ? hold : kManyRows;
  const int form = block > 4 * hold   ? kEight
                   : block > 2 * hold ? kFour
                   : block > hold     ? kTwo
                   : 2 * block > (cache->page_size < many ? cache->page_size : many) ? kOne : kMany;
  a.window = form == kMany ? many / block * block : block;
  // a CTA looks after about one window, or one sequence where those are shorter
  const int mean = cu_seqlens ? (tokens + batch - 1) / batch : 1;
  a.chunk = mean < a.window ? mean : a.window;
  const int64_t chunks = ((int64_t)tokens + a.chunk - 1) / a.chunk;
  // and its warps after several heads, unless that leaves SMs without work
  const int most = by_cta(form) ? 2 * heads_kv : (2 * heads_kv + 3) / 4;
  const int per_sm = (form == kTwo || form == kFour ? 64 : 128) / warps_of(form);
  const int64_t want = (152 * per_sm + chunks - 1) / chunks;
  a.shares = (int)(want < most ? want : most);
  if (chunks * a.shares > 0x7fffffffLL) a.shares = 1;
  const dim3 grid((unsigned)(chunks * a.shares));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (a.err) e = launch_status_clear(a.err, st);
  if (e == cudaSuccess) {
    auto go = [&](auto... kernels) {
      decltype(&append_q8_kernel<__half, kOne, true>) of[] = {kernels...};
      return launch_pdl(of[form], grid, dim3(32 * warps_of(form)), 0, st, a);
    };
    auto typed = [&](auto t, auto full) {
      using T = decltype(t);
      constexpr bool F = decltype(full)::value;
      return go(append_q8_kernel<T, kOne, F>, append_q8_kernel<T, kMany, F>, append_q8_kernel<T, kTwo, F>,
                append_q8_kernel<T, kFour, F>, append_q8_kernel<T, kEight, F>);
    };
    const bool full = a.in_run == 8 && a.out_run == 8;
    if (dtype == SAGE_F16) e = full ? typed(__half{}, std::true_type{}) : typed(__half{}, std::false_type{});
    else e = full ? typed(__nv_bfloat16{}, std::true_type{}) : typed(__nv_bfloat16{}, std::false_type{});
  }
  return e == cudaSuccess ? SAGE_OK : note_cuda_failure(e, "8-bit append");
}

int sage_paged_read_q8(const sage_packed* k_out, const sage_packed* v_out, const sage_q8_cache* cache,
                       const int32_t* cu_seqlens, const int32_t* starts, int batch, int tokens, int heads_kv, int head_dim,
                       int dtype, int tensor_layout, void* workspace, size_t workspace_bytes, void* stream) {
  if (!k_out || !v_out) return SAGE_ERR_INVALID_ARG;
  ReadArgs a{};
  int align = 1;
  int s = make_q8_view(cache, batch, heads_kv, head_dim, tensor_layout, &a.q, &align);
  if (s != SAGE_OK) return s;
  if (dtype != SAGE_F16 && dtype != SAGE_BF16) return SAGE_ERR_DTYPE;
  if (tokens < 0 || !cu_seqlens || reinterpret_cast<uintptr_t>(cu_seqlens) % 4 || reinterpret_cast<uintptr_t>(starts) % 4)
    return SAGE_ERR_INVALID_ARG;
  if (check_status_word(workspace, workspace_bytes) != SAGE_OK) return SAGE_ERR_WORKSPACE;
  if (tokens == 0) return empty_call(workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
  int run = 8;
  const sage_packed* t[2] = {k_out, v_out};
  for (int i = 0; i < 2; ++i) {
    s = check_rows(t[i], tokens, heads_kv, head_dim, true, &run);
    if (s != SAGE_OK) return s;
    a.y[i] = t[i]->data;
    a.y_st[i] = t[i]->stride_token;
    a.y_sh[i] = t[i]->stride_head;
  }
  if (!sage_device_supported()) return SAGE_ERR_DEVICE;
  a.cu = cu_seqlens;
  a.starts = starts;
  a.tokens = tokens;
  a.err = static_cast<int*>(workspace);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (a.err) e = launch_status_clear(a.err, st);
  // rows of a warp: as many as leave some warps for each SM
  const int v = run == 8 && align >= 8 ? 8 : run >= 4 && align >= 4 ? 4 : 1;
  const int runs = heads_kv * ((head_dim + v - 1) / v), most = runs <= 32 ? 8 * (32 / runs) : 4;
  a.rows = tokens / (152 * 16);
  a.rows = a.rows < 1 ? 1 : a.rows > most ? most : a.rows;
  if (a.rows > 32) a.rows = 32;
  const dim3 grid((unsigned)(((int64_t)tokens + 4 * a.rows - 1) / (4 * a.rows)), 2);
  if (e == cudaSuccess) {
    auto go = [&](auto k8, auto k4, auto k1) { return launch_pdl(v == 8 ? k8 : v == 4 ? k4 : k1, grid, dim3(128), 0, st, a); };
    using B = __nv_bfloat16;
    e = dtype == SAGE_F16 ? go(read_q8_kernel<__half, 8>, read_q8_kernel<__half, 4>, read_q8_kernel<__half, 1>)
                          : go(read_q8_kernel<B, 8>, read_q8_kernel<B, 4>, read_q8_kernel<B, 1>);
  }
  return e == cudaSuccess ? SAGE_OK : note_cuda_failure(e, "8-bit read");
}

}  // extern "C"
