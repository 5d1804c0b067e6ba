// Page tables of a paged cache kept on the GPU (sage_paged_assign, sage_paged_release): sequences that grow take pages
// from a stack of free ones, sequences that shrink give theirs back.
//
// Both are prefix sums over the batch and then independent writes, a few microseconds of latency each. A CTA sums what
// comes before its own sequences from the lengths themselves instead of waiting for another CTA, so an assignment is one
// launch; its reads are a few KB that the L2 holds. GPU time: 4.3 us for 256 sequences of one new token, 5.4 for 48 prompts of up
// to 4096 tokens; a release of 256 sequences 4.1, of 64 that an eviction cut 6.4 (two launches each).
#include "../../include/sageattn.h"
#include "launch.h"
#include "paged.cuh"

namespace sage {
namespace {

constexpr int kThreads = 256;

// Sums over the block of two values (every thread gets them).
struct Two {
  long long x, y;
};
__device__ __forceinline__ Two block_sum(Two v) {
  __shared__ Two s[kThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  Two r{0, 0};
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) { r.x += s[w].x; r.y += s[w].y; }
  return r;
}
// Sums of the threads before this one; the block's in `all`.
__device__ __forceinline__ Two block_before(Two v, Two& all) {
  __shared__ Two s[kThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Two inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, inc.x, o), y = __shfl_up_sync(0xffffffffu, inc.y, o);
    if (lane >= o) { inc.x += x; inc.y += y; }
  }
  __syncthreads();
  if (lane == 31) s[warp] = inc;
  __syncthreads();
  Two r{inc.x - v.x, inc.y - v.y};
  all = {0, 0};
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) { r.x += s[w].x; r.y += s[w].y; }
    all.x += s[w].x; all.y += s[w].y;
  }
  return r;
}

// ---------------------------------------------------------------------------------- assignment
struct AssignArgs {
  int* table; int64_t table_stride; int max_pages;
  const int* lens; const int* add; const int* base;  // base: position of the first new token, or null (the length)
  const int* free_pages; const int* free_count; int capacity;
  int batch, page_size, max_tokens;
  int per, splits;  // sequences of a CTA (at most kThreads), CTAs that share them
  int* new_lens; int* held; int* cu; int* positions; long long* slots; int* new_count;
  int* err;         // or null
};

// Tokens and pages of sequence b; `bad`: its length or its new tokens are out of range, or the table has no room.
struct Growth {
  int len, add;
  long long have, need;
  bool bad;
};
__device__ __forceinline__ Growth growth_of(const AssignArgs& a, int b) {
  Growth g{0, 0, 0, 0, false};
  if (b >= a.batch) return g;
  g.len = __ldg(&a.lens[b]);
  g.add = __ldg(&a.add[b]);
  const long long room = (long long)a.max_pages * a.page_size;
  g.bad = g.len < 0 || g.add < 0 || (long long)g.len + g.add > room;
  if (g.add < 0) g.add = 0;
  if (g.bad) return g;
  g.have = ((long long)g.len + a.page_size - 1) / a.page_size;
  g.need = ((long long)g.len + g.add + a.page_size - 1) / a.page_size - g.have;
  return g;
}

// CTA (x, y): sequences [x per, (x + 1) per), share y of their tokens and table entries.
__global__ void __launch_bounds__(kThreads) assign_kernel(const AssignArgs a) {
  __shared__ int s_cu[kThreads + 1], s_len[kThreads], s_served[kThreads];
  __shared__ int s_have[kThreads], s_need[kThreads];
  __shared__ int s_first[kThreads];  // where on the stack the first new page lies
  const int tid = threadIdx.x, b0 = blockIdx.x * a.per, split = blockIdx.y;
  pdl_wait();
  pdl_trigger();
  const int given = __ldg(a.free_count);
  const int count = given < 0 ? 0 : given > a.capacity ? a.capacity : given;
  // tokens and pages of the sequences before this CTA's
  Two before{0, 0};
  for (int b = tid; b < b0; b += kThreads) {
    const Growth g = growth_of(a, b);
    before.x += g.add;
    before.y += g.need;
  }
  before = block_sum(before);
  const int b = b0 + tid;
  const bool mine = tid < a.per && b < a.batch;
  const Growth g = mine ? growth_of(a, b) : Growth{0, 0, 0, 0, false};
  Two all;
  const Two at = block_before({g.add, g.need}, all);
  const long long t0 = before.x + at.x, t1 = t0 + g.add, last = before.y + at.y + g.need;
  const bool bad = g.bad || t1 > a.max_tokens;
  const bool served = mine && !bad && (g.need == 0 || last <= count);
  if (mine) {
    s_cu[tid] = (int)(t0 < a.max_tokens ? t0 : a.max_tokens);
    s_len[tid] = a.base ? __ldg(&a.base[b]) : g.len;
    s_served[tid] = served;
    s_have[tid] = (int)g.have;
    s_need[tid] = served ? (int)g.need : 0;
    s_first[tid] = (int)(count - 1 - (served ? last - g.need : 0));
  }
  const int n = min(a.per, a.batch - b0);
  if (n == 0 && tid == 0) {  // (no sequence at all)
    s_cu[0] = 0;
    if (split == 0) a.cu[0] = 0;
    if (split == 0 && a.err && given != count) record_error(a.err, kDevSeqlens);
  }
  if (tid == n - 1) s_cu[n] = (int)(t1 < a.max_tokens ? t1 : a.max_tokens);
  if (split == 0 && mine) {
    a.cu[b] = s_cu[tid];
    a.new_lens[b] = served ? g.len + g.add : g.len;
    a.held[b] = served ? g.len : -1;
    if (b == a.batch - 1) a.cu[a.batch] = (int)(t1 < a.max_tokens ? t1 : a.max_tokens);
    if (a.err && (bad || given != count)) record_error(a.err, kDevSeqlens);
  }
  __syncthreads();
  // the stack's new height: what the last served sequence that needs pages leaves. The last CTA looks at all of them.
  if (split == 0 && b0 + n == a.batch) {
    long long taken = served && g.need > 0 ? last : 0, sum = 0, tokens = 0;
    for (int i0 = 0; i0 < b0; i0 += kThreads) {
      const Growth o = growth_of(a, i0 + tid < b0 ? i0 + tid : a.batch);
      Two part;
      const Two pre = block_before({o.add, o.need}, part);
      if (!o.bad && o.need > 0 && tokens + pre.x + o.add <= a.max_tokens && sum + pre.y + o.need <= count)
        taken = max(taken, sum + pre.y + o.need);
      tokens += part.x;
      sum += part.y;
    }
    __shared__ unsigned long long s_taken;
    if (tid == 0) s_taken = 0;
    __syncthreads();
    if (taken) atomicMax(&s_taken, (unsigned long long)taken);
    __syncthreads();
    if (tid == 0) *a.new_count = count - (int)s_taken;
  }
  // ---- this CTA's share of the table entries: a warp per sequence
  const int lane = tid & 31, warp = tid >> 5;
  for (int s = warp; s < n; s += kThreads / 32) {
    const int need = s_need[s];
    int* row = a.table + (int64_t)(b0 + s) * a.table_stride + s_have[s];
    for (int i = split * 32 + lane; i < need; i += a.splits * 32) row[i] = __ldg(&a.free_pages[s_first[s] - i]);
  }
  // ---- and of the tokens; behind the last sequence positions and slots are -1
  const int c0 = s_cu[0], c1 = b0 + n == a.batch ? a.max_tokens : s_cu[n];
  for (int64_t t = (int64_t)c0 + split * kThreads + tid; t < c1; t += a.splits * kThreads) {
    long long slot = -1;
    int pos = -1;
    if (t < s_cu[n]) {
      int lo = 0, hi = n - 1;  // the last s with cu[s] <= t
      while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (s_cu[mid] <= t) lo = mid;
        else hi = mid - 1;
      }
      const int i = (int)t - s_cu[lo];
      pos = s_len[lo] + i;
      if (s_served[lo]) {
        const int held = __ldg(&a.lens[b0 + lo]), where = held + i, page = where / a.page_size;
        const int k = page - s_have[lo];
        const int pg = k < 0 ? a.table[(int64_t)(b0 + lo) * a.table_stride + page] : __ldg(&a.free_pages[s_first[lo] - k]);
        if (pg >= 0 && pg < a.capacity) slot = (long long)pg * a.page_size + (where - page * a.page_size);
        else if (a.err) record_error(a.err, kDevPage);
      }
    }
    a.positions[t] = pos;
    a.slots[t] = slot;
  }
}

// ------------------------------------------------------------------------------------- release
struct ReleaseArgs {
  const int* table; int64_t table_stride; int max_pages;
  const int* lens; const int* keep;
  int* free_pages; const int* free_count; int capacity;
  int batch, page_size;
  int* given;      // [batch]: pages of each sequence that go back, or -1 - its error
  int* new_count;
  int* err;
};

__device__ __forceinline__ bool shrink_of(const ReleaseArgs& a, int b, int& keep, int& have) {
  const int len = __ldg(&a.lens[b]), to = __ldg(&a.keep[b]);
  if (to < 0 || to > len || len > (long long)a.max_pages * a.page_size) return false;
  keep = (int)(((long long)to + a.page_size - 1) / a.page_size);
  have = (int)(((long long)len + a.page_size - 1) / a.page_size);
  return true;
}

// A CTA per sequence: how many pages it gives. One with a page that is none gives nothing.
__global__ void __launch_bounds__(kThreads) count_kernel(const ReleaseArgs a) {
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x;
  int keep = 0, have = 0;
  const bool ok = shrink_of(a, b, keep, have);
  bool bad = false;
  for (int i = keep + threadIdx.x; i < have; i += kThreads) {
    const int pg = __ldg(&a.table[(int64_t)b * a.table_stride + i]);
    bad |= pg < 0 || pg >= a.capacity;
  }
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) a.given[b] = !ok ? -1 - kDevSeqlens : bad ? -1 - kDevPage : have - keep;
}

// A CTA per sequence: its pages to their places on the stack. (One CTA where there is no sequence: the count alone.)
__global__ void __launch_bounds__(kThreads) push_kernel(const ReleaseArgs a) {
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x;
  const int said = __ldg(a.free_count);
  const int count = said < 0 ? 0 : said > a.capacity ? a.capacity : said;
  // (x: the pages of the sequences before this one)
  Two sum{0, 0};
  for (int i = threadIdx.x; i < b; i += kThreads) sum.x += max(a.given[i], 0);
  sum = block_sum(sum);
  const int mine = b < a.batch ? max(a.given[b], 0) : 0;
  const bool fits = count + sum.x + mine <= a.capacity;
  if (fits && mine > 0) {
    int keep = 0, have = 0;
    shrink_of(a, b, keep, have);
    for (int i = threadIdx.x; i < mine; i += kThreads)
      a.free_pages[count + sum.x + i] = __ldg(&a.table[(int64_t)b * a.table_stride + keep + i]);
  }
  // the last sequence that fits says how high the stack is: the first CTA finds it, and the status of the call
  if (b == 0) {
    __shared__ unsigned long long s_high;
    __shared__ int s_err;
    if (threadIdx.x == 0) {
      s_high = 0;
      s_err = said != count ? kDevSeqlens : 0;
    }
    __syncthreads();
    long long run = 0;
    for (int i0 = 0; i0 < a.batch; i0 += kThreads) {
      const int i = i0 + threadIdx.x, got = i < a.batch ? a.given[i] : 0, g = max(got, 0);
      Two all;
      const Two at = block_before({g, 0}, all);
      const long long high = run + at.x + g;
      if (got < 0) atomicMax(&s_err, -1 - got);
      else if (g > 0 && count + high <= a.capacity) atomicMax(&s_high, (unsigned long long)high);
      else if (g > 0) atomicMax(&s_err, (int)kDevSeqlens);
      run += all.x;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      *a.new_count = count + (int)s_high;
      if (a.err) *a.err = s_err;
    }
  }
}

// What both calls ask of the table, the lengths and the stack.
int check_tables(const void* table, int64_t stride, int max_pages, const void* lens, const void* other, const void* pages,
                 const void* count, const void* new_count, int num_pages, int page_size, int batch, const void* workspace,
                 size_t workspace_bytes, size_t need) {
  auto off = [](const void* p) { return !p || reinterpret_cast<uintptr_t>(p) % 4; };
  if (batch < 0 || batch > 65535 || num_pages < 0 || page_size < 1 || max_pages < 0 || stride < 0 ||
      (int64_t)max_pages * page_size > kMostSlots)
    return SAGE_ERR_INVALID_ARG;
  if (off(count) || off(new_count) || count == new_count) return SAGE_ERR_INVALID_ARG;
  if (num_pages > 0 && off(pages)) return SAGE_ERR_INVALID_ARG;
  if (batch > 0 && (off(lens) || off(other) || (max_pages > 0 && off(table)))) return SAGE_ERR_INVALID_ARG;
  if (batch > 1 && stride < max_pages) return SAGE_ERR_STRIDE;  // rows that share entries
  if (workspace ? reinterpret_cast<uintptr_t>(workspace) % 256 || workspace_bytes < need : need > SAGE_STATUS_BYTES)
    return SAGE_ERR_WORKSPACE;
  return SAGE_OK;
}

}  // namespace
}  // namespace sage

using namespace sage;

extern "C" {

int sage_paged_assign(int32_t* page_table, int64_t table_stride, int max_pages, const int32_t* seq_lens,
                      const int32_t* add_lens, const int32_t* next_positions, const int32_t* free_pages,
                      const int32_t* free_count, int num_pages, int page_size, int batch, int max_tokens,
                      int32_t* new_lens, int32_t* held_lens, int32_t* cu_seqlens, int32_t* positions, int64_t* slots,
                      int32_t* new_free_count, void* workspace, size_t workspace_bytes, void* stream) {
  const int s = check_tables(page_table, table_stride, max_pages, seq_lens, add_lens, free_pages, free_count,
                             new_free_count, num_pages, page_size, batch, workspace, workspace_bytes, SAGE_STATUS_BYTES);
  if (s != SAGE_OK) return s;
  auto off = [](const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; };
  if (max_tokens < 0 || !cu_seqlens || off(cu_seqlens, 4) || off(next_positions, 4)) return SAGE_ERR_INVALID_ARG;
  if (batch > 0 && (!new_lens || !held_lens || off(new_lens, 4) || off(held_lens, 4))) return SAGE_ERR_INVALID_ARG;
  if (max_tokens > 0 && (!positions || !slots || off(positions, 4) || off(slots, 8))) return SAGE_ERR_INVALID_ARG;
  // (the lengths are read while the results are written)
  const uintptr_t span = (uintptr_t)batch * 4;
  for (const void* in : {(const void*)seq_lens, (const void*)add_lens, (const void*)next_positions})
    for (const void* out : {(const void*)new_lens, (const void*)held_lens})
      if (in && out && reinterpret_cast<uintptr_t>(in) < reinterpret_cast<uintptr_t>(out) + span &&
          reinterpret_cast<uintptr_t>(out) < reinterpret_cast<uintptr_t>(in) + span)
        return SAGE_ERR_INVALID_ARG;
  if (!sage_device_supported()) return SAGE_ERR_DEVICE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  AssignArgs a{};
  a.table = page_table; a.table_stride = table_stride; a.max_pages = max_pages;
  a.lens = seq_lens; a.add = add_lens; a.base = next_positions;
  a.free_pages = free_pages; a.free_count = free_count; a.capacity = num_pages;
  a.batch = batch; a.page_size = page_size; a.max_tokens = max_tokens;
  a.new_lens = new_lens; a.held = held_lens; a.cu = cu_seqlens; a.positions = positions;
  a.slots = reinterpret_cast<long long*>(slots);
  a.new_count = new_free_count;
  a.err = static_cast<int*>(workspace);
  cudaError_t e = cudaSuccess;
  if (a.err) e = launch_status_clear(a.err, st);
  // as many sequences per CTA as leave a CTA for each SM; those of long rows share their tokens
  a.per = (batch + 151) / 152;
  a.per = a.per < 1 ? 1 : a.per > kThreads ? kThreads : a.per;
  const int groups = batch > 0 ? (batch + a.per - 1) / a.per : 1;
  const int64_t share = max_tokens / groups / 1024;
  a.splits = (int)(share < 1 ? 1 : share > 128 ? 128 : share);
  if (e == cudaSuccess) e = launch_pdl(assign_kernel, dim3(groups, a.splits), dim3(kThreads), 0, st, a);
  return e == cudaSuccess ? SAGE_OK : note_cuda_failure(e, "page assignment");
}

size_t sage_paged_release_workspace_size(int batch) {
  return batch < 0 || batch > 65535 ? 0 : SAGE_STATUS_BYTES + ((size_t)batch * 4 + 255) / 256 * 256;
}

int sage_paged_release(const int32_t* page_table, int64_t table_stride, int max_pages, const int32_t* seq_lens,
                       const int32_t* keep_lens, int32_t* free_pages, const int32_t* free_count, int num_pages,
                       int page_size, int batch, int32_t* new_free_count, void* workspace, size_t workspace_bytes,
                       void* stream) {
  const int s = check_tables(page_table, table_stride, max_pages, seq_lens, keep_lens, free_pages, free_count,
                             new_free_count, num_pages, page_size, batch, workspace, workspace_bytes,
                             sage_paged_release_workspace_size(batch));
  if (s != SAGE_OK) return s;
  if (!workspace && batch > 0) return SAGE_ERR_WORKSPACE;
  if (!sage_device_supported()) return SAGE_ERR_DEVICE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  ReleaseArgs a{};
  a.table = page_table; a.table_stride = table_stride; a.max_pages = max_pages;
  a.lens = seq_lens; a.keep = keep_lens;
  a.free_pages = free_pages; a.free_count = free_count; a.capacity = num_pages;
  a.batch = batch; a.page_size = page_size;
  a.given = batch > 0 ? reinterpret_cast<int*>(static_cast<char*>(workspace) + SAGE_STATUS_BYTES) : nullptr;
  a.new_count = new_free_count;
  a.err = static_cast<int*>(workspace);
  cudaError_t e = cudaSuccess;
  if (batch > 0) e = launch_pdl(count_kernel, dim3(batch), dim3(kThreads), 0, st, a);
  if (e == cudaSuccess) e = launch_pdl(push_kernel, dim3(batch > 0 ? batch : 1), dim3(kThreads), 0, st, a);
  return e == cudaSuccess ? SAGE_OK : note_cuda_failure(e, "page release");
}

}  // extern "C"
