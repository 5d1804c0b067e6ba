// Filling and thinning a paged key-value cache: sage_paged_append writes new tokens into their pages,
// sage_paged_evict keeps each (sequence, head)'s most attended tokens.
#include <cmath>

#include "launch.h"
#include "paged.cuh"
#include "sm103_ptx.cuh"

namespace sage {

int make_paged_view(const sage_paged_cache* c, int batch, int heads_kv, int head_dim, int dtype, int layout,
                    PagedView* view, bool* vec) {
  if (!c) return SAGE_ERR_INVALID_ARG;
  if (head_dim < 1 || head_dim > 128) return SAGE_ERR_HEAD_DIM;
  if (dtype != SAGE_F16 && dtype != SAGE_BF16) return SAGE_ERR_DTYPE;
  if (layout != SAGE_HND && layout != SAGE_NHD) return SAGE_ERR_INVALID_ARG;
  if (batch < 0 || heads_kv < 1 || heads_kv > 65535 || c->num_pages < 0 || c->page_size < 1 || c->max_pages < 0 ||
      (int64_t)c->max_pages * c->page_size > kMostSlots)
    return SAGE_ERR_INVALID_ARG;
  PagedView v{};
  v.batch = batch; v.hkv = heads_kv; v.d = head_dim;
  v.page_size = c->page_size; v.num_pages = c->num_pages; v.max_pages = c->max_pages;
  if (batch > 0) {
    auto off = [](const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; };
    if ((!c->page_table && c->max_pages > 0) || !c->seq_lens || off(c->page_table, 4) || off(c->seq_lens, 4) || off(c->mass, 4) ||
        off(c->positions, 4) || c->table_stride < 0)
      return SAGE_ERR_INVALID_ARG;
    if (c->num_pages > 0 && (!c->k || !c->v)) return SAGE_ERR_INVALID_ARG;
    if (off(c->k, 2) || off(c->v, 2)) return SAGE_ERR_STRIDE;
    for (int i = 0; i < 3; ++i)
      if (c->k_stride[i] < 0 || c->v_stride[i] < 0) return SAGE_ERR_STRIDE;
  }
  const int hi = layout == SAGE_HND ? 1 : 2, ti = layout == SAGE_HND ? 2 : 1;
  v.k = c->k; v.k_sp = c->k_stride[0]; v.k_sh = c->k_stride[hi]; v.k_st = c->k_stride[ti];
  v.v = c->v; v.v_sp = c->v_stride[0]; v.v_sh = c->v_stride[hi]; v.v_st = c->v_stride[ti];
  v.table = c->page_table; v.table_stride = c->table_stride; v.lens = c->seq_lens;
  v.mass = c->mass; v.pos = c->positions;
  bool w = head_dim % 8 == 0 && reinterpret_cast<uintptr_t>(c->k) % 16 == 0 && reinterpret_cast<uintptr_t>(c->v) % 16 == 0;
  for (int i = 0; i < 3; ++i) w = w && c->k_stride[i] % 8 == 0 && c->v_stride[i] % 8 == 0;
  *view = v;
  *vec = w;
  return SAGE_OK;
}

namespace {

// ------------------------------------------------------------------------------------- append
struct AppendArgs {
  PagedView c;
  const uint16_t* k; int64_t k_st, k_sh;
  const uint16_t* v; int64_t v_st, v_sh;
  const int* cu;        // [batch + 1] or null: one token per sequence
  const int* new_pos;   // [tokens] or null: the slot
  int tokens, vec;
  int* err;             // or null
};

// One warp per token: the token's sequence by bisection of cu_seqlens, its slot and page, then its K
// and V rows of every head, 16 bytes per lane. Memory-bound for prompts; for one token per sequence the chain of
// dependent loads (length, page, row) is what it costs. 16 prompts of 1K to 4K tokens: 57.6 us, 95% of a copy's rate; 64 sequences
// of one token: 2.4 us. A 16-bit pattern is copied whatever its type.
__global__ void __launch_bounds__(128) append_kernel(const AppendArgs a) {
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * 4 + (threadIdx.x >> 5);
  pdl_wait();
  if (t >= a.tokens) return;
  int b = t, at = 0;
  if (a.cu) {
    int lo = 0, hi = a.c.batch;  // the last b with cu[b] <= t
    while (hi - lo > 0) {
      const int mid = lo + (hi - lo + 1) / 2;
      if (__ldg(&a.cu[mid]) <= t) lo = mid;
      else hi = mid - 1;
    }
    b = lo;
    const int first = __ldg(&a.cu[b]);
    if (a.err && t == 0 && lane == 0 && first != 0) record_error(a.err, kDevSeqlens);
    if (b == a.c.batch || first > t) return;  // behind the last sequence, or before the first
    at = t - first;
  }
  const int held = __ldg(&a.c.lens[b]);
  const int64_t slot = (int64_t)held + at;
  // (a negative length refuses all of its tokens: the later ones would land on slots in use)
  if (held < 0 || slot >= (int64_t)a.c.max_pages * a.c.page_size) {
    if (a.err && lane == 0) record_error(a.err, kDevSeqlens);
    return;
  }
  const int i = (int)(slot / a.c.page_size), sl = (int)(slot - (int64_t)i * a.c.page_size);
  const int page = __ldg(&a.c.table[b * a.c.table_stride + i]);
  if (page < 0 || page >= a.c.num_pages) {
    if (a.err && lane == 0) record_error(a.err, kDevPage);
    return;
  }
  const uint16_t* ks = a.k + t * a.k_st;
  const uint16_t* vs = a.v + t * a.v_st;
  uint16_t* kd = static_cast<uint16_t*>(a.c.k) + page * a.c.k_sp + sl * a.c.k_st;
  uint16_t* vd = static_cast<uint16_t*>(a.c.v) + page * a.c.v_sp + sl * a.c.v_st;
  if (a.vec) {
    const int nch = a.c.d / 8, n = a.c.hkv * nch;
#pragma unroll 4
    for (int x = lane; x < n; x += 32) {
      const int h = x / nch, c = (x - h * nch) * 8;
      const uint4 kx = __ldg(reinterpret_cast<const uint4*>(ks + h * a.k_sh + c));
      const uint4 vx = __ldg(reinterpret_cast<const uint4*>(vs + h * a.v_sh + c));
      *reinterpret_cast<uint4*>(kd + h * a.c.k_sh + c) = kx;
      *reinterpret_cast<uint4*>(vd + h * a.c.v_sh + c) = vx;
    }
  } else {
    for (int x = lane; x < a.c.hkv * a.c.d; x += 32) {
      const int h = x / a.c.d, c = x - h * a.c.d;
      kd[h * a.c.k_sh + c] = ks[h * a.k_sh + c];
      vd[h * a.c.v_sh + c] = vs[h * a.v_sh + c];
    }
  }
  if (a.c.mass || a.c.pos) {
    const int p = a.new_pos ? __ldg(&a.new_pos[t]) : (int)slot;
    for (int h = lane; h < a.c.hkv; h += 32) {
      const int64_t w = plane_at(a.c, page, h, sl);
      if (a.c.mass) a.c.mass[w] = 0.f;
      if (a.c.pos) a.c.pos[w] = p;
    }
  }
}

__global__ void status_clear_kernel(int* err) {
  pdl_wait();
  *err = 0;
}

}  // namespace

cudaError_t launch_status_clear(int* err, cudaStream_t st) {
  return launch_pdl(status_clear_kernel, dim3(1), dim3(1), 0, st, err);
}

int empty_call(void* workspace, size_t workspace_bytes, cudaStream_t st) {
  // (nothing is asked of the workspace of a call that has nothing to do: it need be no memory of the device, nor must there be one)
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 || workspace_bytes < SAGE_STATUS_BYTES) return SAGE_OK;
  if (!sage_device_supported()) return SAGE_OK;
  cudaPointerAttributes at{};
  if (cudaPointerGetAttributes(&at, workspace) != cudaSuccess) {
    cudaGetLastError();
    return SAGE_OK;
  }
  if (at.type != cudaMemoryTypeDevice && at.type != cudaMemoryTypeManaged) return SAGE_OK;
  const cudaError_t e = launch_status_clear(static_cast<int*>(workspace), st);
  return e == cudaSuccess ? SAGE_OK : note_cuda_failure(e, "status reset");
}

namespace {

// ---------------------------------------------------------------------------------- eviction
struct EvictArgs {
  PagedView c;
  int budget, sink, recent, max_len, vec;
  int page_shift;  // log2 of page_size, or -1
  int cached;      // codes that the selection's shared memory holds
  int vec4;        // four slots lie in one page and in aligned 16 bytes of the planes
  int* new_lens;
  int* block_err;  // [batch * hkv]
  int* err;
  int* count;      // [batch * hkv]: tokens that move
  int* to;         // [batch * hkv][pitch]: freed slots below the budget, ascending
  int* from;       // [batch * hkv][pitch]: kept slots from the budget on, ascending
  int64_t pitch;
};

constexpr int kSelThreads = 1024;
constexpr int kBins = 2048;

// A weight's order as an unsigned code: NaN last (with -inf), both zeros alike.
__device__ __forceinline__ unsigned weight_code(float w) {
  return ordered_code(isnan(w) ? -INFINITY : w + 0.0f);
}

// Sum over the block of x and the exclusive prefix of this thread.
__device__ __forceinline__ int block_scan(int x, int& total) {
  __shared__ int s[kSelThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  __syncthreads();
  if (lane == 31) s[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    int v = s[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    s[lane] = v;
  }
  __syncthreads();
  total = s[kSelThreads / 32 - 1];
  return inc - x + (warp ? s[warp - 1] : 0);
}

// Words of another CTA of the cluster.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ int ld_rank(const int* p, int rank) {
  int v;
  asm volatile(
      "{\n\t.reg .u32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.u32 %0, [a];\n\t}"
      : "=r"(v)
      : "r"(smem_u32(p)), "r"(rank)
      : "memory");
  return v;
}

// One CTA per (head, sequence), or a cluster of R, each with a stretch of the slots. The budget-th largest weight is found by a radix selection over the
// ordered codes (three digits of 11, 11 and 10 bits, one histogram each: integer counts, so the
// result does not depend on any order); then the slots are walked in order, ties taken from the
// lowest slot on, and the freed slots below the budget and the kept ones behind it are listed.
// A pass over the planes is a chain of two dependent loads per slot (page, then value), so they are read once
// each with eight slots per thread in flight, and the codes stay in shared memory for the passes of
// the selection, which read four at a time. (A sequence with more tokens than fit is read again, in
// chunks, by each pass.) 64 heads of 6000 to 32768 tokens, cut to 4096: 26 us here by clusters of two (33 by one CTA each), then
// 37 to move the rows, which is 75% of a copy's rate; the selection is bound by the latency of its passes.
constexpr int kAhead = 8;
constexpr int kMostCached = 48 * 1024;
template <int R>
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a) {
  extern __shared__ __align__(16) unsigned codes[];  // of `cached` slots; 0: no token
  __shared__ int hist[kBins];
  __shared__ int s_pick, s_rest, s_last, s_bad;
  __shared__ int s_cnt[32][4];
  __shared__ int s_give[4];  // what the other CTAs of the cluster read
  const int rank = R > 1 ? (int)(blockIdx.x % R) : 0;
  const int h = blockIdx.x / R, b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t me = (int64_t)b * a.c.hkv + h;
  pdl_wait();
  const int len = checked_len(a.c, b, a.max_len);
  if (tid == 0) { s_last = INT32_MIN; s_bad = len < 0 ? kDevSeqlens : 0; }
  for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
  __syncthreads();
  const int keep = a.budget;
  if (len <= keep) {  // nothing to drop (or a length that is refused)
    if (tid == 0 && rank == 0) {
      a.count[me] = 0;
      a.block_err[me] = s_bad;
      if (h == 0) a.new_lens[b] = a.c.lens[b];
    }
    return;
  }
  const int per = ((len + R - 1) / R + 3) & ~3;
  const int begin = min(len, rank * per), stop = min(len, begin + per);  // this CTA's slots
  const int* table = a.c.table + b * a.c.table_stride;
  // Plane indexes of eight groups of slots, the first of group u at j0 + u G kSelThreads, or -1 (behind `end`; or
  // on a bad page, which sets `bad`). A group is the G slots of one thread, in one page. Pages are loaded
  // for all groups before any is looked at: with a branch between, each waits for the last.
  bool bad = false;
  auto where = [&](auto g, int j0, int end, int64_t (&w)[kAhead]) {
    constexpr int G = decltype(g)::value;
    int pg[kAhead], sl[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead / G; ++u) {
      const int j = min(j0 + u * G * kSelThreads, len - 1);
      const int i = a.page_shift >= 0 ? j >> a.page_shift : j / a.c.page_size;
      sl[u] = j - i * a.c.page_size;
      pg[u] = __ldg(&table[i]);
    }
#pragma unroll
    for (int u = 0; u < kAhead / G; ++u) {
      const bool in = pg[u] >= 0 && pg[u] < a.c.num_pages;
      bad = bad || !in;
      w[u] = in && j0 + u * G * kSelThreads < end ? plane_at(a.c, pg[u], h, sl[u]) : -1;
    }
  };
  // eight positions or weights of a thread; x where there is none (behind `end` within a group: any)
  auto take = [&](auto g, const auto* plane, const int64_t (&w)[kAhead], auto x, auto (&v)[kAhead]) {
    constexpr int G = decltype(g)::value;
#pragma unroll
    for (int u = 0; u < kAhead / G; ++u) {
      if constexpr (G == 4) {
        int4 q = make_int4(0, 0, 0, 0);
        if (w[u] >= 0) q = *reinterpret_cast<const int4*>(plane + w[u]);
        const int t[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if constexpr (std::is_same<decltype(x), float>::value) v[u * 4 + k] = __int_as_float(t[k]);
          else v[u * 4 + k] = t[k];
        }
      } else {
        v[u] = w[u] >= 0 ? plane[w[u]] : x;
      }
    }
  };
  auto newest = [&](auto g) {
    constexpr int G = decltype(g)::value;
    int last = INT32_MIN;
    for (int j0 = begin + tid * G; j0 < stop; j0 += kSelThreads * kAhead) {
      int64_t w[kAhead];
      int p[kAhead];
      where(g, j0, stop, w);
      take(g, a.c.pos, w, INT32_MIN, p);
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (w[u / G] >= 0 && j0 + (u / G) * G * kSelThreads + u % G < stop) last = max(last, p[u]);
    }
    return last;
  };
  using One = std::integral_constant<int, 1>;
  using Four = std::integral_constant<int, 4>;
  {
    const int last = __reduce_max_sync(0xffffffffu, a.vec4 ? newest(Four{}) : newest(One{}));
    if (lane == 0) atomicMax(&s_last, last);
    if (bad) s_bad = kDevPage;
  }
  __syncthreads();
  int newest_pos = s_last, wrong = s_bad;
  if constexpr (R > 1) {
    if (tid < 2) s_give[tid] = tid == 0 ? s_last : s_bad;
    cluster_sync();
    for (int i = 0; i < R; ++i) {
      newest_pos = max(newest_pos, ld_rank(&s_give[0], i));
      wrong = max(wrong, ld_rank(&s_give[1], i));
    }
    cluster_sync();
  }
  if (h == 0 && rank == 0 && tid == 0) a.new_lens[b] = wrong ? len : keep;  // (every head reads the same pages)
  if (wrong) {
    if (tid == 0 && rank == 0) { a.count[me] = 0; a.block_err[me] = wrong; }
    return;
  }
  const int64_t recent_from = (int64_t)newest_pos - a.recent;
  const int cap = a.cached;  // a multiple of 4
  const bool once = R > 1 || len <= cap;  // (clusters: the host saw to it)
  // codes of the slots [c0, c0 + cap); their first digit is counted with `count`
  auto load_group = [&](auto g, int c0, int n, bool count) {
    constexpr int G = decltype(g)::value;
    const int end = min(c0 + n, stop);
    for (int j0 = tid * G; j0 < n; j0 += kSelThreads * kAhead) {
      int64_t w[kAhead];
      int p[kAhead];
      float x[kAhead];
      where(g, c0 + j0, end, w);
      take(g, a.c.pos, w, 0, p);
      take(g, a.c.mass, w, 0.f, x);
      unsigned c[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int j = j0 + (u / G) * G * kSelThreads + u % G;
        c[u] = w[u / G] < 0 || c0 + j >= end                  ? 0u
               : p[u] < a.sink || (int64_t)p[u] > recent_from ? 0xFFFFFFFFu
                                                              : weight_code(x[u]);
        if (count && c[u]) atomicAdd(&hist[c[u] >> 21], 1);
      }
#pragma unroll
      for (int u = 0; u < kAhead / G; ++u) {
        const int j = j0 + u * G * kSelThreads;
        if (j < n) {
          if constexpr (G == 4) *reinterpret_cast<uint4*>(&codes[j]) = make_uint4(c[4 * u], c[4 * u + 1], c[4 * u + 2], c[4 * u + 3]);
          else codes[j] = c[u];
        }
      }
    }
  };
  auto load_codes = [&](int c0, bool count) {
    const int n = min(cap, (stop - c0 + 3) & ~3);
    if (a.vec4) load_group(Four{}, c0, n, count);
    else load_group(One{}, c0, n, count);
    return n;
  };
  int loaded = 0;
  if (once) {
    loaded = load_codes(begin, true);
    __syncthreads();
  }
  unsigned prefix = 0, mask = 0;
  int rest = keep;  // how many of the codes that match the prefix are kept
#pragma unroll 1
  for (int digit = 0; digit < 3; ++digit) {
    const int shift = digit == 0 ? 21 : digit == 1 ? 10 : 0, bins = digit == 2 ? 1024 : 2048;
    if (digit > 0) {
      for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
      __syncthreads();
    }
    if (digit > 0 || !once)
      for (int c0 = begin; c0 < stop; c0 += cap) {
        const int n = once ? loaded : load_codes(c0, digit == 0);
        if (!once) __syncthreads();
        if (digit > 0)
          for (int j = tid * 4; j < n; j += kSelThreads * 4) {
            const uint4 c = *reinterpret_cast<const uint4*>(&codes[j]);
            if ((c.x & mask) == prefix) atomicAdd(&hist[(c.x >> shift) & (bins - 1)], 1);
            if ((c.y & mask) == prefix) atomicAdd(&hist[(c.y >> shift) & (bins - 1)], 1);
            if ((c.z & mask) == prefix) atomicAdd(&hist[(c.z >> shift) & (bins - 1)], 1);
            if ((c.w & mask) == prefix) atomicAdd(&hist[(c.w >> shift) & (bins - 1)], 1);
          }
        __syncthreads();
      }
    // bins from the top: the one in which the rest-th largest lies
    const int hi = kBins - 1 - 2 * tid;
    int x1 = hist[hi], x0 = hist[hi - 1];
    if constexpr (R > 1) {
      cluster_sync();
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (i != rank) {
          x1 += ld_rank(&hist[hi], i);
          x0 += ld_rank(&hist[hi - 1], i);
        }
      cluster_sync();
    }
    int total;
    const int before = block_scan(x1 + x0, total);
    if (before < rest && rest <= before + x1) { s_pick = hi; s_rest = rest - before; }
    else if (before + x1 < rest && rest <= before + x1 + x0) { s_pick = hi - 1; s_rest = rest - before - x1; }
    __syncthreads();
    prefix |= (unsigned)s_pick << shift;
    mask |= (unsigned)(bins - 1) << shift;
    rest = s_rest;
    __syncthreads();
  }
  // The threshold is `prefix`; of the slots that equal it the first `rest` are kept. In each chunk a warp walks its
  // own stretch, four slots per lane: first what it holds below and behind the budget is counted, which
  // gives every warp its place in the lists, then the lists are written.
  int* to = a.to + me * a.pitch;
  int* from = a.from + me * a.pitch;
  int ties = 0, holes = 0, movers = 0;  // before this chunk
  int c0 = begin;
  do {
    const int n = once ? loaded : load_codes(c0, false);
    if (!once) __syncthreads();
    const int span = (n + 32 * 128 - 1) / (32 * 128) * 128;
    const int j_lo = min(n, warp * span), j_hi = min(n, j_lo + span);
    int over_lo = 0, over_hi = 0, tie_lo = 0, tie_hi = 0;
    for (int j = j_lo + lane * 4; j < j_hi; j += 128) {
      const uint4 v = *reinterpret_cast<const uint4*>(&codes[j]);
      const unsigned c[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const bool low = c0 + j + u < keep;
        over_lo += c[u] > prefix && low;
        over_hi += c[u] > prefix && !low;
        tie_lo += c[u] == prefix && low;
        tie_hi += c[u] == prefix && !low;
      }
    }
    over_lo = __reduce_add_sync(0xffffffffu, over_lo);
    over_hi = __reduce_add_sync(0xffffffffu, over_hi);
    tie_lo = __reduce_add_sync(0xffffffffu, tie_lo);
    tie_hi = __reduce_add_sync(0xffffffffu, tie_hi);
    if (lane == 0) {
      s_cnt[warp][0] = over_lo; s_cnt[warp][1] = over_hi;
      s_cnt[warp][2] = tie_lo; s_cnt[warp][3] = tie_hi;
    }
    __syncthreads();
    if constexpr (R > 1) {
      // what the CTAs before this one hold
      if (warp < 4) {
        const int x = __reduce_add_sync(0xffffffffu, s_cnt[lane][warp]);
        if (lane == 0) s_give[warp] = x;
      }
      cluster_sync();
      for (int i = 0; i < rank; ++i) {
        const int o_lo = ld_rank(&s_give[0], i), o_hi = ld_rank(&s_give[1], i);
        const int t_lo = ld_rank(&s_give[2], i), t_hi = ld_rank(&s_give[3], i);
        const int kept_lo = min(t_lo, max(0, rest - ties)), kept_hi = min(t_hi, max(0, rest - ties - t_lo));
        const int low = max(0, min(min(len, (i + 1) * per), keep) - i * per);
        ties += t_lo + t_hi;
        holes += low - o_lo - kept_lo;
        movers += o_hi + kept_hi;
      }
    }
    // the sums over the warps before this one, and over all for the next chunk: lane w has warp w's counts
    const int o_lo = s_cnt[lane][0], o_hi = s_cnt[lane][1], t_lo = s_cnt[lane][2], t_hi = s_cnt[lane][3];
    const int w_lo = min(n, lane * span), w_hi = min(n, w_lo + span);
    const int low = max(0, min(min(c0 + w_hi, keep), stop) - (c0 + w_lo));  // its slots below the budget
    int t_sum = t_lo + t_hi;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, t_sum, o);
      if (lane >= o) t_sum += x;
    }
    const int t_before = ties + t_sum - t_lo - t_hi;
    const int kept_lo = min(t_lo, max(0, rest - t_before)), kept_hi = min(t_hi, max(0, rest - t_before - t_lo));
    const int my_h = low - o_lo - kept_lo, my_m = o_hi + kept_hi;
    int h_sum = my_h, m_sum = my_m;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, h_sum, o), y = __shfl_up_sync(0xffffffffu, m_sum, o);
      if (lane >= o) { h_sum += x; m_sum += y; }
    }
    int my_ties = __shfl_sync(0xffffffffu, t_before, warp);
    int my_holes = holes + __shfl_sync(0xffffffffu, h_sum - my_h, warp);
    int my_movers = movers + __shfl_sync(0xffffffffu, m_sum - my_m, warp);
    ties += __shfl_sync(0xffffffffu, t_sum, 31);
    holes += __shfl_sync(0xffffffffu, h_sum, 31);
    movers += __shfl_sync(0xffffffffu, m_sum, 31);
    const unsigned lower = (1u << lane) - 1u;
    for (int j0 = j_lo; j0 < j_hi; j0 += 128) {
      const int j = j0 + lane * 4;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (j < j_hi) v = *reinterpret_cast<const uint4*>(&codes[j]);
      const unsigned c[4] = {v.x, v.y, v.z, v.w};
      int tie = my_ties;  // ties before this lane's slots
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const unsigned t = __ballot_sync(0xffffffffu, c[u] == prefix);
        tie += __popc(t & lower);
        my_ties += __popc(t);
      }
      bool hole[4], mover[4];
      int at_h = my_holes, at_m = my_movers;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const bool kept = c[u] > prefix || (c[u] == prefix && tie < rest), low = c0 + j + u < keep;
        tie += c[u] == prefix;
        hole[u] = c[u] != 0 && low && !kept;
        mover[u] = kept && !low;
        const unsigned bh = __ballot_sync(0xffffffffu, hole[u]), bm = __ballot_sync(0xffffffffu, mover[u]);
        at_h += __popc(bh & lower);
        at_m += __popc(bm & lower);
        my_holes += __popc(bh);
        my_movers += __popc(bm);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (hole[u]) to[at_h++] = c0 + j + u;
        if (mover[u]) from[at_m++] = c0 + j + u;
      }
    }
    __syncthreads();
    c0 += cap;
  } while (c0 < stop);
  if (tid == 0 && rank == R - 1) { a.count[me] = movers; a.block_err[me] = 0; }
  if constexpr (R > 1) cluster_sync();  // no CTA's shared memory goes away while it is read
}

// Moves the listed tokens: a half warp per token, 16 bytes per lane. Sources lie behind the budget and
// targets below it, so no move reads what another one writes. (More tokens in flight per half warp measured
// slower, since the registers cost resident warps: 2 and 4 of them 11 and 15 us more for 64 heads of up to 32K tokens, whose
// moves take 37.)
__global__ void __launch_bounds__(256, 8) evict_move_kernel(const EvictArgs a) {
  const int h = blockIdx.y, b = blockIdx.z;
  const int64_t me = (int64_t)b * a.c.hkv + h;
  pdl_wait();
  if (blockIdx.x == 0 && h == 0 && b == 0) {
    int e = 0;
    for (int i = threadIdx.x; i < a.c.batch * a.c.hkv; i += 256) e = max(e, a.block_err[i]);
    e = __reduce_max_sync(0xffffffffu, e);
    __shared__ int s_e[8];
    if ((threadIdx.x & 31) == 0) s_e[threadIdx.x >> 5] = e;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int i = 0; i < 8; ++i) e = max(e, s_e[i]);
      *a.err = e;
    }
  }
  const int n = a.count[me];
  const int* table = a.c.table + b * a.c.table_stride;
  const int lane = threadIdx.x & 15;
  uint16_t* kb = static_cast<uint16_t*>(a.c.k) + h * a.c.k_sh;
  uint16_t* vb = static_cast<uint16_t*>(a.c.v) + h * a.c.v_sh;
  for (int i = blockIdx.x * 16 + (threadIdx.x >> 4); i < n; i += gridDim.x * 16) {
    const int to = a.to[me * a.pitch + i], from = a.from[me * a.pitch + i];
    const int ti = to / a.c.page_size, fi = from / a.c.page_size;
    const int ts = to - ti * a.c.page_size, fs = from - fi * a.c.page_size;
    const int tp = __ldg(&table[ti]), fp = __ldg(&table[fi]);
    const uint16_t* ks = kb + fp * a.c.k_sp + fs * a.c.k_st;
    const uint16_t* vs = vb + fp * a.c.v_sp + fs * a.c.v_st;
    uint16_t* kd = kb + tp * a.c.k_sp + ts * a.c.k_st;
    uint16_t* vd = vb + tp * a.c.v_sp + ts * a.c.v_st;
    if (a.vec) {
      if (lane * 8 < a.c.d) {
        const uint4 kx = *reinterpret_cast<const uint4*>(ks + lane * 8);
        const uint4 vx = *reinterpret_cast<const uint4*>(vs + lane * 8);
        *reinterpret_cast<uint4*>(kd + lane * 8) = kx;
        *reinterpret_cast<uint4*>(vd + lane * 8) = vx;
      }
    } else {
      for (int c = lane; c < a.c.d; c += 16) {
        kd[c] = ks[c];
        vd[c] = vs[c];
      }
    }
    if (lane == 0) {
      const int64_t wt = plane_at(a.c, tp, h, ts), wf = plane_at(a.c, fp, h, fs);
      a.c.mass[wt] = a.c.mass[wf];
      a.c.pos[wt] = a.c.pos[wf];
    }
  }
}

// The selection by clusters of R for at most `most` slots per CTA (R == 1: more are read in chunks).
template <int R>
cudaError_t launch_select(EvictArgs a, int most, int heads_kv, cudaStream_t st) {
  a.cached = most < kMostCached ? (most + 3) / 4 * 4 : kMostCached;
  static std::atomic<int> limits[64];
  const cudaError_t e = raise_smem_limit(evict_select_kernel<R>, kMostCached * 4, limits);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(heads_kv * R, a.c.batch);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = (size_t)a.cached * 4;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = R;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = R > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, evict_select_kernel<R>, a);
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }
struct EvictLayout {
  size_t block_err, count, to, from, total;
  int64_t pitch;
};
// A (sequence, head) moves at most min(budget, max_seqlen - budget) tokens.
bool evict_layout(int batch, int hkv, int max_len, int budget, EvictLayout* L) {
  if (batch < 0 || hkv < 1 || max_len < 0 || budget < 0) return false;
  const int64_t most = max_len > budget ? (budget < max_len - budget ? budget : max_len - budget) : 0;
  L->pitch = most;
  const size_t n = (size_t)batch * hkv;
  size_t o = 256;
  auto take = [&](size_t bytes) { const size_t at = o; o += up256(bytes); return at; };
  L->block_err = take(4 * n);
  L->count = take(4 * n);
  L->to = take(4 * n * most);
  L->from = take(4 * n * most);
  L->total = o;
  return true;
}

}  // namespace
}  // namespace sage

using namespace sage;

extern "C" {

int sage_paged_append(const sage_packed* k, const sage_packed* v, const sage_paged_cache* cache,
                      const int32_t* cu_seqlens, const int32_t* positions, int batch, int tokens, int heads_kv,
                      int head_dim, int dtype, int tensor_layout, void* workspace, size_t workspace_bytes,
                      void* stream) {
  if (!k || !v || !cache) return SAGE_ERR_INVALID_ARG;
  AppendArgs a{};
  bool vec = false;
  const int s = make_paged_view(cache, batch, heads_kv, head_dim, dtype, tensor_layout, &a.c, &vec);
  if (s != SAGE_OK) return s;
  if (tokens < 0 || (!cu_seqlens && tokens != batch)) return SAGE_ERR_INVALID_ARG;
  if (workspace && (reinterpret_cast<uintptr_t>(workspace) % 256 || workspace_bytes < SAGE_STATUS_BYTES))
    return SAGE_ERR_WORKSPACE;
  if (batch == 0 || tokens == 0) return empty_call(workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
  if (!k->data || !v->data || reinterpret_cast<uintptr_t>(cu_seqlens) % 4 || reinterpret_cast<uintptr_t>(positions) % 4)
    return SAGE_ERR_INVALID_ARG;
  for (const sage_packed* t : {k, v}) {
    if (reinterpret_cast<uintptr_t>(t->data) % 2 || t->stride_token < 0 || t->stride_head < 0) return SAGE_ERR_STRIDE;
    vec = vec && reinterpret_cast<uintptr_t>(t->data) % 16 == 0 && t->stride_token % 8 == 0 && t->stride_head % 8 == 0;
  }
  if (!sage_device_supported()) return SAGE_ERR_DEVICE;
  a.k = static_cast<const uint16_t*>(k->data); a.k_st = k->stride_token; a.k_sh = k->stride_head;
  a.v = static_cast<const uint16_t*>(v->data); a.v_st = v->stride_token; a.v_sh = v->stride_head;
  a.cu = cu_seqlens;
  a.new_pos = positions;
  a.tokens = tokens;
  a.vec = vec ? 1 : 0;
  a.err = static_cast<int*>(workspace);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (a.err) e = launch_status_clear(a.err, st);
  if (e == cudaSuccess) e = launch_pdl(append_kernel, dim3((unsigned)(((int64_t)tokens + 3) / 4)), dim3(128), 0, st, a);
  return e == cudaSuccess ? SAGE_OK : note_cuda_failure(e, "paged append");
}

size_t sage_paged_evict_workspace_size(int batch, int heads_kv, int max_seqlen, int budget) {
  EvictLayout L;
  return evict_layout(batch, heads_kv, max_seqlen, budget, &L) ? L.total : 0;
}

int sage_paged_evict(const sage_paged_cache* cache, int32_t* new_lens, int batch, int heads_kv, int max_seqlen,
                     int head_dim, int dtype, int tensor_layout, int budget, int sink, int recent, void* workspace,
                     size_t workspace_bytes, void* stream) {
  if (!cache) return SAGE_ERR_INVALID_ARG;
  EvictArgs a{};
  bool vec = false;
  const int s = make_paged_view(cache, batch, heads_kv, head_dim, dtype, tensor_layout, &a.c, &vec);
  if (s != SAGE_OK) return s;
  if (max_seqlen < 0 || batch > 65535 || budget < 1 || sink < 0 || recent < 0 || (int64_t)sink + recent > budget)
    return SAGE_ERR_INVALID_ARG;
  if (batch == 0) return empty_call(workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
  // (planes of no pages have no address, and are not read)
  if (!new_lens || reinterpret_cast<uintptr_t>(new_lens) % 4 || (cache->num_pages > 0 && (!cache->mass || !cache->positions)))
    return SAGE_ERR_INVALID_ARG;
  // (seq_lens is read by the CTAs of every head, after the first has written new_lens)
  const uintptr_t n0 = reinterpret_cast<uintptr_t>(new_lens), l0 = reinterpret_cast<uintptr_t>(cache->seq_lens);
  if (n0 < l0 + 4 * (size_t)batch && l0 < n0 + 4 * (size_t)batch) return SAGE_ERR_INVALID_ARG;
  EvictLayout L;
  if (!evict_layout(batch, heads_kv, max_seqlen, budget, &L)) return SAGE_ERR_INVALID_ARG;
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 || workspace_bytes < L.total)
    return SAGE_ERR_WORKSPACE;
  if (!sage_device_supported()) return SAGE_ERR_DEVICE;
  char* w = static_cast<char*>(workspace);
  a.budget = budget; a.sink = sink; a.recent = recent; a.max_len = max_seqlen; a.vec = vec ? 1 : 0;
  a.new_lens = new_lens;
  a.err = reinterpret_cast<int*>(w);
  a.block_err = reinterpret_cast<int*>(w + L.block_err);
  a.count = reinterpret_cast<int*>(w + L.count);
  a.to = reinterpret_cast<int*>(w + L.to);
  a.from = reinterpret_cast<int*>(w + L.from);
  a.pitch = L.pitch;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  a.page_shift = -1;
  for (int i = 0; i < 31; ++i)
    if (cache->page_size == 1 << i) a.page_shift = i;
  a.vec4 = cache->page_size % 4 == 0 && reinterpret_cast<uintptr_t>(cache->mass) % 16 == 0 &&
           reinterpret_cast<uintptr_t>(cache->positions) % 16 == 0;
  // Few heads with long sequences: clusters, so that more SMs read and count (1024 threads fill an SM's registers). Their
  // barriers and sums cost 5 to 8 us, so one CTA is faster up to some 18K tokens. us per call of 8 heads, nothing moved, by
  // one CTA, clusters of two and of four: 4096 tokens 10.5, 15.1, 18.0; 16384 18.1, 18.8, 19.9; 32768 28.8, 24.1, 22.2
  // (64 heads: 29.2, 24.6, 45.1, where clusters of four no longer run at once).
  const int64_t heads = (int64_t)batch * heads_kv;
  const int ranks = max_seqlen <= 18432 ? 1 : heads * 4 <= 152 ? 4 : heads * 2 <= 152 ? 2 : 1;
  const int share = (max_seqlen + ranks - 1) / ranks;
  cudaError_t e = ranks == 4 && share <= kMostCached - 4   ? launch_select<4>(a, share, heads_kv, st)
                  : ranks == 2 && share <= kMostCached - 4 ? launch_select<2>(a, share, heads_kv, st)
                                                           : launch_select<1>(a, max_seqlen, heads_kv, st);
  // enough CTAs to fill the GPU, none that could not have work
  int64_t blocks = (L.pitch + 15) / 16, most = 1216 / ((int64_t)batch * heads_kv);
  blocks = blocks < 1 ? 1 : blocks;
  most = most < 1 ? 1 : most;
  if (e == cudaSuccess)
    e = launch_pdl(evict_move_kernel, dim3((unsigned)(blocks < most ? blocks : most), heads_kv, batch), dim3(256), 0, st, a);
  return e == cudaSuccess ? SAGE_OK : note_cuda_failure(e, "paged eviction");
}

}  // extern "C"
