// Filling an 8-bit paged key-value cache and taking its values out again (sage_paged_append_q8, sage_paged_read_q8).
//
// The scale of a block follows its tokens: the largest magnitude among them decides it (needed_scale). A token that joins
// a block whose scale is too small raises the scale to what it needs, and the codes of the block's earlier tokens are
// rounded again to the new one: for E4M3 that moves an exponent and is exact but for subnormals; for int8 it adds at most
// half a step for each time a block's scale grows, which for tokens of one distribution is a few times in a block.
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

// The sequence of row t, the last b with cu[b] <= t (batch: behind the last one).
__device__ __forceinline__ int sequence_of(const int* cu, int batch, int t) {
  int lo = 0, hi = batch;
  while (lo < hi) {
    const int mid = lo + (hi - lo + 1) / 2;
    if (__ldg(&cu[mid]) <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// ------------------------------------------------------------------------------------- append
struct AppendArgs {
  Q8View q;
  const void* x[2]; int64_t x_st[2], x_sh[2];  // k, v: element strides of token and head
  const int* cu;        // [batch + 1] or null: one token per sequence
  int tokens, chunk;    // rows that a CTA looks after
  int in16, out8;       // rows allow 16-byte loads, codes 8-byte stores
  int lanes;            // lanes of a row, 8 channels each: 8 or 16
  int* err;             // or null
};

// The rows of one block and head: their largest magnitude, the scale, the codes. WARPS warps share a block.
template <typename T, int TYPE, int WARPS>
__device__ __forceinline__ void store_block(const AppendArgs& a, int kv, int h, int64_t row0, int rows, int page, int slot0,
                                            bool joins) {
  constexpr int kKept = 8;  // rows per lane that stay in registers between the two walks
  __shared__ float s_most[4];
  const int lane = threadIdx.x & 31, warp = WARPS == 1 ? 0 : threadIdx.x >> 5;
  const PagedView& c = a.q.c;
  const int ch = (lane & (a.lanes - 1)) * 8, per = 32 / a.lanes, step = per * WARPS;
  const int first = warp * per + lane / a.lanes;
  const bool on = ch < c.d;
  const T* x = static_cast<const T*>(a.x[kv]) + row0 * a.x_st[kv] + h * a.x_sh[kv];
  const int64_t xs = a.x_st[kv];
  uint8_t* base = static_cast<uint8_t*>(kv ? c.v : c.k) + page * (kv ? c.v_sp : c.k_sp) + h * (kv ? c.v_sh : c.k_sh);
  const int64_t cs = kv ? c.v_st : c.k_st;
  float* const scales = kv ? a.q.vs : a.q.ks;
  const int64_t at = scale_at(a.q, page, h, slot0);
  const int held = slot0 % a.q.block;  // earlier tokens of the block, where it is joined
  const float was = joins ? scales[at] : 0.f;
  uint4 kept[kKept];
  float most = 0.f;
#pragma unroll
  for (int i = 0; i < kKept; ++i) {
    kept[i] = make_uint4(0, 0, 0, 0);
    const int r = first + i * step;
    if (on && r < rows) kept[i] = load8_raw<T>(x + r * xs, ch, c.d, a.in16);
  }
#pragma unroll
  for (int i = 0; i < kKept; ++i) {
    const T* t = reinterpret_cast<const T*>(&kept[i]);
#pragma unroll
    for (int e = 0; e < 8; ++e) most = fmaxf(most, fabsf(to_f32<T>(t[e])));
  }
  for (int r = first + kKept * step; r < rows; r += step) {
    float y[8];
    if (on) {
      load8<T>(x + r * xs, ch, c.d, a.in16, y);
#pragma unroll
      for (int e = 0; e < 8; ++e) most = fmaxf(most, fabsf(y[e]));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
  if (WARPS > 1) {
    __syncthreads();  // (also: every thread has read the old scale)
    if (lane == 0) s_most[warp] = most;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WARPS; ++w) most = fmaxf(most, s_most[w]);
  }
  const float scale = fmaxf(was, needed_scale<TYPE>(most)), inv = __frcp_rn(scale);
  __syncwarp();  // (every lane has read the old scale)
  if (threadIdx.x % (32 * WARPS) == 0) scales[at] = scale;
  auto put = [&](int slot, const uint8_t (&code)[8]) {
    uint8_t* d = base + slot * cs + ch;
    if (a.out8 && ch + 8 <= c.d) {
      *reinterpret_cast<uint2*>(d) = *reinterpret_cast<const uint2*>(code);
    } else {
      for (int e = 0; e < 8; ++e)
        if (ch + e < c.d) d[e] = code[e];
    }
  };
  if (joins && scale > was) {
    const float f = __fdiv_rn(was, scale);
    for (int r = first; r < held; r += step) {
      if (!on) break;
      const int slot = slot0 - held + r;
      const uint8_t* s = base + slot * cs + ch;
      alignas(8) uint8_t code[8];
      if (a.out8 && ch + 8 <= c.d) {
        *reinterpret_cast<uint2*>(code) = *reinterpret_cast<const uint2*>(s);
      } else {
        for (int e = 0; e < 8; ++e) code[e] = ch + e < c.d ? s[e] : 0;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) code[e] = to_code<TYPE>(from_code<TYPE>(code[e]) * f);
      put(slot, code);
    }
  }
  auto write = [&](int r, const float (&y)[8]) {
    alignas(8) uint8_t code[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) code[e] = to_code<TYPE>(y[e] * inv);
    put(slot0 + r, code);
  };
#pragma unroll
  for (int i = 0; i < kKept; ++i) {
    const int r = first + i * step;
    if (!on || r >= rows) continue;
    const T* t = reinterpret_cast<const T*>(&kept[i]);
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = to_f32<T>(t[e]);
    write(r, y);
  }
  for (int r = first + kKept * step; r < rows; r += step) {
    if (!on) break;
    float y[8];
    load8<T>(x + r * xs, ch, c.d, a.in16, y);
    write(r, y);
  }
}

// CTA (x, y): the blocks whose first new token lies in rows [x chunk, (x + 1) chunk), for one of the heads' K or V
// (WARPS 4: the CTA shares a block; 1: each of its four warps takes another head or side).
template <typename T, int WARPS>
__global__ void __launch_bounds__(128) append_q8_kernel(const AppendArgs a) {
  const PagedView& c = a.q.c;
  const int unit = WARPS == 4 ? blockIdx.y : blockIdx.y * 4 + (threadIdx.x >> 5);
  const int h = unit >> 1, kv = unit & 1;
  pdl_wait();
  pdl_trigger();
  if (h >= c.hkv) return;  // (a whole warp, or no thread of the CTA)
  const bool tells = a.err && unit == 0 && (threadIdx.x & 31) == 0 && (WARPS == 1 || threadIdx.x == 0);
  const int64_t t_end = min((int64_t)a.tokens, ((int64_t)blockIdx.x + 1) * a.chunk);
  int64_t t = (int64_t)blockIdx.x * a.chunk;
  int b = a.cu ? sequence_of(a.cu, c.batch, (int)t) : (int)t;
  while (t < t_end) {
    int64_t first = t, end = t + 1;
    if (a.cu) {
      first = __ldg(&a.cu[b]);
      if (tells && t == 0 && first != 0) record_error(a.err, kDevSeqlens);
      if (b >= c.batch) return;              // behind the last sequence
      if (first > t) return;                 // before the first
      end = min((int64_t)__ldg(&a.cu[b + 1]), (int64_t)a.tokens);
      if (end <= t) { ++b; continue; }       // a sequence without tokens (b grows: at most batch of them)
    }
    const int len = __ldg(&c.lens[b]);
    const int64_t room = (int64_t)c.max_pages * c.page_size;
    const int64_t slot = (int64_t)len + t - first;
    if (len < 0 || slot >= room) {
      if (tells) record_error(a.err, kDevSeqlens);
      t = end;                               // the rest of this sequence
      if (a.cu) ++b;
      else b = (int)t;
      continue;
    }
    const int in = (int)(slot % a.q.block);
    int64_t next = min(end, t + a.q.block - in);
    if (t == first || in == 0) {             // the first new token of its block
      const int i = (int)(slot / c.page_size), s0 = (int)(slot - (int64_t)i * c.page_size);
      const int page = __ldg(&c.table[b * c.table_stride + i]);
      if (page < 0 || page >= c.num_pages) {
        if (tells) record_error(a.err, kDevPage);
      } else if (kv == 0) {
        if (a.q.k_type == SAGE_S8) store_block<T, SAGE_S8, WARPS>(a, 0, h, t, (int)(next - t), page, s0, in != 0);
        else store_block<T, SAGE_E4M3, WARPS>(a, 0, h, t, (int)(next - t), page, s0, in != 0);
      } else {
        if (a.q.v_type == SAGE_S8) store_block<T, SAGE_S8, WARPS>(a, 1, h, t, (int)(next - t), page, s0, in != 0);
        else store_block<T, SAGE_E4M3, WARPS>(a, 1, h, t, (int)(next - t), page, s0, in != 0);
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
  int tokens;
  int* err;
};

template <int TYPE, int V>
__device__ __forceinline__ void decode(const uint8_t* p, float scale, float (&y)[V]) {
  alignas(16) uint8_t code[V];
  if constexpr (V == 16) *reinterpret_cast<uint4*>(code) = __ldg(reinterpret_cast<const uint4*>(p));
  else if constexpr (V == 8) *reinterpret_cast<uint2*>(code) = __ldg(reinterpret_cast<const uint2*>(p));
  else code[0] = *p;
#pragma unroll
  for (int e = 0; e < V; ++e) y[e] = from_code<TYPE>(code[e]) * scale;
}
template <typename T>
__device__ __forceinline__ T narrow(float x) {
  if constexpr (std::is_same<T, __half>::value) return __float2half_rn(x);
  else return __float2bfloat16_rn(x);
}

// A warp per row of the result: V codes per lane and access, the heads one after the other.
template <typename T, int V>
__global__ void __launch_bounds__(128) read_q8_kernel(const ReadArgs a) {
  const PagedView& c = a.q.c;
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  pdl_wait();
  pdl_trigger();
  if (t >= a.tokens) return;
  const int b = sequence_of(a.cu, c.batch, (int)t);
  int page = -1, slot = 0;
  const int first = __ldg(&a.cu[b]);
  if (a.err && t == 0 && lane == 0 && first != 0) record_error(a.err, kDevSeqlens);
  if (b < c.batch && first <= t) {
    const int len = __ldg(&c.lens[b]);
    const int64_t s = (a.starts ? __ldg(&a.starts[b]) : 0) + t - first;
    const int64_t room = (int64_t)c.max_pages * c.page_size;
    if (s < 0 || s >= len || s >= room) {
      if (a.err && lane == 0) record_error(a.err, kDevSeqlens);
    } else {
      const int i = (int)(s / c.page_size);
      slot = (int)(s - (int64_t)i * c.page_size);
      page = __ldg(&c.table[b * c.table_stride + i]);
      if (page < 0 || page >= c.num_pages) {
        page = -1;
        if (a.err && lane == 0) record_error(a.err, kDevPage);
      }
    }
  }
  const int runs = (c.d + V - 1) / V, n = c.hkv * runs;
  for (int x = lane; x < 2 * n; x += 32) {
    const int kv = x >= n, y = x - kv * n, h = y / runs, ch = (y - h * runs) * V;
    alignas(16) T out[V];
    if (page >= 0) {
      const uint8_t* p = static_cast<const uint8_t*>(kv ? c.v : c.k) + page * (kv ? c.v_sp : c.k_sp) + h * (kv ? c.v_sh : c.k_sh) +
                         slot * (kv ? c.v_st : c.k_st) + ch;
      const float scale = __ldg((kv ? a.q.vs : a.q.ks) + scale_at(a.q, page, h, slot));
      float f[V];
      if ((kv ? a.q.v_type : a.q.k_type) == SAGE_S8) decode<SAGE_S8, V>(p, scale, f);
      else decode<SAGE_E4M3, V>(p, scale, f);
#pragma unroll
      for (int e = 0; e < V; ++e) out[e] = narrow<T>(f[e]);
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) out[e] = T(0.0f);
    }
    T* dst = static_cast<T*>(a.y[kv]) + t * a.y_st[kv] + h * a.y_sh[kv] + ch;
    if constexpr (V >= 8) {
#pragma unroll
      for (int e = 0; e < V; e += 8) *reinterpret_cast<uint4*>(dst + e) = *reinterpret_cast<const uint4*>(out + e);
    } else {
      dst[0] = out[0];
    }
  }
}

__global__ void clear_status_kernel(int* err) {
  pdl_wait();
  *err = 0;
}

int check_status_word(const void* workspace, size_t bytes) {
  return workspace && (reinterpret_cast<uintptr_t>(workspace) % 256 || bytes < SAGE_STATUS_BYTES) ? SAGE_ERR_WORKSPACE
                                                                                                 : SAGE_OK;
}
// A packed operand of rows; *vec: every row of whole 16-byte accesses.
int check_rows(const sage_packed* t, int tokens, int heads, int d, bool written, bool* vec) {
  if (!t->data) return SAGE_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(t->data) % 2 || t->stride_token < 0 || t->stride_head < 0) return SAGE_ERR_STRIDE;
  if (written && ((tokens > 1 && t->stride_token == 0) || (heads > 1 && t->stride_head == 0))) return SAGE_ERR_STRIDE;
  *vec = *vec && reinterpret_cast<uintptr_t>(t->data) % 16 == 0 && d % 8 == 0 && (tokens <= 1 || t->stride_token % 8 == 0) &&
         (heads <= 1 || t->stride_head % 8 == 0);
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
  if (batch == 0 || tokens == 0) return SAGE_OK;
  bool vec = true;
  const sage_packed* t[2] = {k, v};
  for (int i = 0; i < 2; ++i) {
    s = check_rows(t[i], tokens, heads_kv, head_dim, false, &vec);
    if (s != SAGE_OK) return s;
    a.x[i] = t[i]->data;
    a.x_st[i] = t[i]->stride_token;
    a.x_sh[i] = t[i]->stride_head;
  }
  if (!sage_device_supported()) return SAGE_ERR_DEVICE;
  a.cu = cu_seqlens;
  a.tokens = tokens;
  a.in16 = vec;
  a.out8 = align >= 8;
  a.lanes = head_dim <= 64 ? 8 : 16;
  a.err = static_cast<int*>(workspace);
  // a CTA looks after about one block, or one sequence where those are shorter
  const int mean = cu_seqlens ? (tokens + batch - 1) / batch : 1, most = a.q.block > 16 ? a.q.block : 16;
  a.chunk = mean < most ? mean : most;
  const int64_t chunks = ((int64_t)tokens + a.chunk - 1) / a.chunk;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (a.err) e = launch_pdl(clear_status_kernel, dim3(1), dim3(1), 0, st, a.err);
  const bool shared = a.chunk > 16;
  const dim3 grid((unsigned)chunks, shared ? 2 * heads_kv : (2 * heads_kv + 3) / 4);
  if (e == cudaSuccess) {
    if (dtype == SAGE_F16)
      e = shared ? launch_pdl(append_q8_kernel<__half, 4>, grid, dim3(128), 0, st, a)
                 : launch_pdl(append_q8_kernel<__half, 1>, grid, dim3(128), 0, st, a);
    else
      e = shared ? launch_pdl(append_q8_kernel<__nv_bfloat16, 4>, grid, dim3(128), 0, st, a)
                 : launch_pdl(append_q8_kernel<__nv_bfloat16, 1>, grid, dim3(128), 0, st, a);
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
  if (tokens == 0) return SAGE_OK;
  bool vec = true;
  const sage_packed* t[2] = {k_out, v_out};
  for (int i = 0; i < 2; ++i) {
    s = check_rows(t[i], tokens, heads_kv, head_dim, true, &vec);
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
  if (a.err) e = launch_pdl(clear_status_kernel, dim3(1), dim3(1), 0, st, a.err);
  const dim3 grid((unsigned)(((int64_t)tokens + 3) / 4));
  const int v = vec && align >= 16 ? 16 : vec && align >= 8 ? 8 : 1;
  if (e == cudaSuccess) {
    auto go = [&](auto k16, auto k8, auto k1) {
      return launch_pdl(v == 16 ? k16 : v == 8 ? k8 : k1, grid, dim3(128), 0, st, a);
    };
    e = dtype == SAGE_F16 ? go(read_q8_kernel<__half, 16>, read_q8_kernel<__half, 8>, read_q8_kernel<__half, 1>)
                          : go(read_q8_kernel<__nv_bfloat16, 16>, read_q8_kernel<__nv_bfloat16, 8>,
                               read_q8_kernel<__nv_bfloat16, 1>);
  }
  return e == cudaSuccess ? SAGE_OK : note_cuda_failure(e, "8-bit read");
}

}  // extern "C"
