// What the decode kernels over a paged cache share: the line of (sequence, head, key tile) items and its ranges, pages,
// fragments, clusters, and the kernel that joins results that lie in several ranges.
#pragma once
#include <cmath>

#include "paged.cuh"
#include "sm103_ptx.cuh"

namespace sage {
namespace {

constexpr int kWarps = 4;
constexpr int kCtas = 304;                 // two resident CTAs per SM: the most of the clusters' form, ranges of the 16-bit line
constexpr int kRows = 16;                  // query heads per row block
constexpr int kMinTiles = 2;               // tiles a CTA takes at least
constexpr int kRanks = 8;                  // CTAs of a cluster
enum { kLoadTma = 0, kLoadVec = 1, kLoadAny = 2 };
constexpr float kLog2eF = 1.4426950408889634f, kLn2F = 0.6931471805599453f;

struct DecodeArgs {
  PagedView c;
  const void* q; int64_t q_sb, q_sh;
  void* o; int64_t o_sb, o_sh;
  float* lse;               // [batch, hq] or null
  const float* slopes;      // [hq] or null
  const int* q_pos;         // [batch] or null (length - 1)
  float sm_scale, cap;
  int hq, group, row_blocks, max_len;
  int load;                 // how rows are read: kLoadTma, kLoadVec or kLoadAny
  int box_rows;             // rows of a TMA box
  int page_shift;           // log2 of page_size, or -1
  int mass4;                // four slots of the mass plane lie in one page and in aligned 16 bytes
  int slices;               // CTAs of the join per (row block of a head, sequence)
  int tile_shift;           // log2 of a tile's keys
  int side;                 // key/value heads that share an item of the line
  int part_rows;            // rows of a piece
  // workspace
  int* err;                 // status word, or null (no workspace: the clusters' form without mass)
  int* cta_err;             // [ranges]: one word for each CTA of the line, whose number is the kernel's own
  float* part_o;            // [ranges][2][side][part_rows][dp]
  float* part_ml;           // [ranges][2][side][part_rows][2], or [4] with FRAMES
  float* lse2;              // [batch, hq], base 2 (with mass)
  float* scores;            // [batch, hq, score_pitch], base 2 (with mass) or null
  int64_t score_pitch;
};

// Tiles of 2^shift keys of a sequence of n tokens.
__device__ __forceinline__ int tiles_of(int n, int shift) {
  return (n + (1 << shift) - 1) >> shift;
}
__host__ __device__ constexpr int log2_of(int x) { return x <= 1 ? 0 : 1 + log2_of(x / 2); }

// The items (sequence, head, tile) of sequences [b0, b0 + blockDim): this thread's count, the sum before it and the
// sum of all. Lengths that are out of range count as 0 and set `bad`.
struct Scan {
  long long n, before, all;
};
__device__ __forceinline__ Scan scan_items(const DecodeArgs& a, int shift, int heads, int b0, bool& bad) {
  __shared__ long long s_sum[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const int b = b0 + threadIdx.x;
  Scan r{0, 0, 0};
  if (b < a.c.batch) {
    const int len = checked_len(a.c, b, a.max_len);
    if (len < 0) bad = true;
    r.n = (long long)tiles_of(max(len, 0), shift) * heads;
  }
  long long inc = r.n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  __syncthreads();
  if (lane == 31) s_sum[warp] = inc;
  __syncthreads();
  r.before = inc - r.n;
  for (int w = 0; w < nw; ++w) {
    if (w < warp) r.before += s_sum[w];
    r.all += s_sum[w];
  }
  return r;
}

// CTAs that share `total` items, and the first item of CTA i.
template <int CTAS>
__device__ __forceinline__ int ctas_of(long long total) {
  const long long g = (total + kMinTiles - 1) / kMinTiles;
  return (int)(g < CTAS ? g : CTAS);
}
__device__ __forceinline__ long long first_item(long long total, int ctas, int i) {
  return total * i / ctas;
}

// One place on the line of items.
struct Cursor {
  int b, h, tile, tiles, len;  // h: head * row_blocks + row block
};
__device__ __forceinline__ void next_item(const DecodeArgs& a, int shift, int heads, Cursor& u) {
  if (++u.tile < u.tiles) return;
  u.tile = 0;
  if (++u.h < heads) return;
  u.h = 0;
  do {
    ++u.b;
    u.len = u.b < a.c.batch ? max(checked_len(a.c, u.b, a.max_len), 0) : 0;
  } while (u.b < a.c.batch && u.len == 0);
  u.tiles = tiles_of(u.len, shift);
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
template <typename T>
__device__ __forceinline__ T round_to(float x) {
  if constexpr (std::is_same<T, __half>::value) return __float2half_rn(x);
  else return __float2bfloat16_rn(x);
}

__device__ __forceinline__ int page_index(const DecodeArgs& a, int key) {
  return a.page_shift >= 0 ? key >> a.page_shift : key / a.c.page_size;
}
// Page and slot of token `key` of sequence b; page -1 where there is none.
__device__ __forceinline__ void find_page(const DecodeArgs& a, int b, int key, bool live, int& page, int& slot, int& err) {
  page = -1;
  slot = 0;
  if (!live) return;
  const int i = page_index(a, key);
  slot = key - i * a.c.page_size;
  const int pg = __ldg(&a.c.table[b * a.c.table_stride + i]);
  if (pg >= 0 && pg < a.c.num_pages) page = pg;
  else err = kDevPage;
}

__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

// Waits for a stage's TMA boxes, two seconds at most.
__device__ __forceinline__ bool wait_stage(uint32_t bar, uint32_t parity) {
  unsigned long long t0 = 0;
  for (uint32_t it = 0; it < (1u << 30); ++it) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(1000u)
        : "memory");
    if (ok) return true;
    if ((it & 63u) == 63u) {
      const unsigned long long t = global_timer_ns();
      if (t0 == 0) t0 = t;
      else if (t - t0 > kWaitTimeoutNs) return false;
    }
  }
  return false;
}

// ---- few heads: a cluster per (sequence, row block of a head), joined through distributed shared memory
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t of_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float2 ld_rank2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_rank4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

// ------------------------------------------------------------------------------------- join
// One CTA per (row block of a head, sequence), or per 32 of its channels: the results that lie in several ranges summed in
// the order of the ranges; sequences that hold nothing get 0 and -inf. CTA (0, 0) also collects the status. FRAMES: a
// piece's accumulator has a frame of its own besides that of the sum of its weights.
constexpr int kJoinThreads = 256;

template <typename T, int DP, int CTAS, bool FRAMES = false>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const DecodeArgs a) {
  __shared__ float s_w[CTAS][kRows];       // weight of each range's piece
  __shared__ int s_at[CTAS];               // and its first row
  __shared__ float s_m[kRows], s_l[kRows], s_f[kRows];
  __shared__ __align__(16) float s_acc[kJoinThreads * 4];
  __shared__ long long s_before[kJoinThreads / 32], s_all[kJoinThreads / 32];
  const int heads = a.c.hkv / a.side * a.row_blocks;
  const int hb = blockIdx.x / a.slices, slice = blockIdx.x - hb * a.slices;
  const int b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // The lengths are older than the decode kernel, which waited for what wrote them before it let this one begin (as it did
  // before it let a kernel begin that another host thread has put between them): what follows from them is found while the
  // decode kernel still runs.
  auto collect = [&]() {  // the status of the call
    if (blockIdx.x > 0 || b > 0) return;
    int e = 0;
    for (int i = tid; i < CTAS; i += kJoinThreads) e = max(e, a.cta_err[i]);
    e = __reduce_max_sync(0xffffffffu, e);
    __syncthreads();
    if (lane == 0) s_all[warp] = e;
    __syncthreads();
    if (tid == 0) {
      for (int w = 0; w < kJoinThreads / 32; ++w) e = max(e, (int)s_all[w]);
      *a.err = e;
    }
  };
  // items before this sequence, and in all
  long long before = 0, all = 0;
  for (int i = tid; i < a.c.batch; i += kJoinThreads) {
    const long long n = (long long)tiles_of(max(checked_len(a.c, i, a.max_len), 0), a.tile_shift) * heads;
    all += n;
    if (i < b) before += n;
  }
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) {
    all += __shfl_xor_sync(0xffffffffu, all, w);
    before += __shfl_xor_sync(0xffffffffu, before, w);
  }
  if (lane == 0) { s_before[warp] = before; s_all[warp] = all; }
  __syncthreads();
  before = all = 0;
  for (int w = 0; w < kJoinThreads / 32; ++w) { before += s_before[w]; all += s_all[w]; }

  const int len = max(checked_len(a.c, b, a.max_len), 0);
  const int h = hb / a.row_blocks, rb = hb - h * a.row_blocks;
  const int row0 = h * a.group + rb * kRows, rows = min(kRows, a.group - rb * kRows);
  if (len == 0) {
    pdl_wait();
    pdl_trigger();
    collect();
    if (slice > 0) return;
    for (int i = tid; i < rows * a.c.d; i += kJoinThreads) {
      const int r = i / a.c.d, c = i - r * a.c.d;
      static_cast<T*>(a.o)[b * a.o_sb + (row0 + r) * a.o_sh + c] = T(0.0f);
    }
    if (a.lse && tid < rows) a.lse[(int64_t)b * a.hq + row0 + tid] = -INFINITY;
    return;
  }
  const int item = h / a.side * a.row_blocks + rb, sub = h % a.side;
  const long long t0 = before + (long long)item * tiles_of(len, a.tile_shift), t1 = t0 + tiles_of(len, a.tile_shift);
  const int ctas = ctas_of<CTAS>(all);
  // the ranges that hold t0 and t1 - 1: range i is [all i / ctas, all (i + 1) / ctas)
  auto range_of = [&](long long t) { return (int)(((t + 1) * ctas - 1) / all); };
  const int c0 = range_of(t0), c1 = range_of(t1 - 1);
  if (c0 == c1) {  // written by its own range
    pdl_wait();
    pdl_trigger();
    collect();
    return;
  }
  const int parts = c1 - c0 + 1;
  // a range's first piece is this one's unless it starts before it
  for (int p = tid; p < parts; p += kJoinThreads) 
    s_at[p] = (((c0 + p) * 2 + (first_item(all, ctas, c0 + p) < t0 ? 1 : 0)) * a.side + sub) * a.part_rows;
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  // accumulators, four channels per thread; threads left over take every n-th piece. The first pieces are fetched
  // while the statistics are
  constexpr int kAhead = 4;
  const int groups = DP / 4 / a.slices, cells = rows * groups;  // groups of four channels
  const int sets = cells >= kJoinThreads ? 1 : kJoinThreads / cells;
  const int set = sets > 1 ? tid / cells : 0;
  float4 x[kAhead];
  auto fetch = [&](int base) {
    const int cell = sets > 1 ? tid - set * cells : base + tid;
    if (set >= sets || cell >= cells) return;
    const int r = cell / groups, c = (slice * groups + cell - r * groups) * 4;
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (set + i * sets < parts) x[i] = *reinterpret_cast<const float4*>(a.part_o + ((int64_t)s_at[set + i * sets] + r) * DP + c);
  };
  fetch(0);
  // row statistics: one warp per row
  for (int r = warp; r < rows; r += kJoinThreads / 32) {
    constexpr int kStats = FRAMES ? 4 : 2;
    float m = -INFINITY, f = -INFINITY;
    for (int p = lane; p < parts; p += 32) {
      m = fmaxf(m, a.part_ml[(s_at[p] + r) * kStats]);
      if (FRAMES) f = fmaxf(f, a.part_ml[(s_at[p] + r) * kStats + 2]);
    }
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) {
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
      if (FRAMES) f = fmaxf(f, __shfl_xor_sync(0xffffffffu, f, w));
    }
    const float u = m == -INFINITY ? 0.f : m, fu = f == -INFINITY ? 0.f : f;
    float l = 0.f;
    for (int p = lane; p < parts; p += 32) {
      const float2 y = *reinterpret_cast<const float2*>(a.part_ml + (s_at[p] + r) * kStats);
      const float w = ex2_approx(y.x - u);
      s_w[p][r] = FRAMES ? ex2_approx(a.part_ml[(s_at[p] + r) * kStats + 2] - fu) : w;
      l += y.y * w;
    }
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) l += __shfl_xor_sync(0xffffffffu, l, w);
    if (lane == 0) {
      s_m[r] = m;
      s_l[r] = l;
      if (FRAMES) s_f[r] = l != 0.f ? ex2_approx(fu - u) / l : 0.f;
    }
  }
  __syncthreads();
  for (int base = 0; base < cells; base += kJoinThreads) {
    const int cell = sets > 1 ? tid - set * cells : base + tid;
    const bool on = set < sets && cell < cells;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    const int r = on ? cell / groups : 0, c = (slice * groups + (on ? cell - r * groups : 0)) * 4;
    if (base > 0) fetch(base);
    if (on) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (set + i * sets < parts) {
          const float w = s_w[set + i * sets][r];
          acc.x = fmaf(w, x[i].x, acc.x); acc.y = fmaf(w, x[i].y, acc.y);
          acc.z = fmaf(w, x[i].z, acc.z); acc.w = fmaf(w, x[i].w, acc.w);
        }
#pragma unroll 8
      for (int p = set + kAhead * sets; p < parts; p += sets) {
        const float4 y = *reinterpret_cast<const float4*>(a.part_o + ((int64_t)s_at[p] + r) * DP + c);
        const float w = s_w[p][r];
        acc.x = fmaf(w, y.x, acc.x); acc.y = fmaf(w, y.y, acc.y);
        acc.z = fmaf(w, y.z, acc.z); acc.w = fmaf(w, y.w, acc.w);
      }
    }
    if (sets > 1) {
      *reinterpret_cast<float4*>(&s_acc[tid * 4]) = acc;
      __syncthreads();
      if (tid < cells)
        for (int s = 1; s < sets; ++s) {
          const float4 y = *reinterpret_cast<const float4*>(&s_acc[(s * cells + tid) * 4]);
          acc.x += y.x; acc.y += y.y; acc.z += y.z; acc.w += y.w;
        }
    }
    if (on && set == 0) {
      const float inv = FRAMES ? s_f[r] : s_l[r] != 0.f ? 1.0f / s_l[r] : 0.f;
      T* dst = static_cast<T*>(a.o) + b * a.o_sb + (row0 + r) * a.o_sh + c;
      const float y[4] = {acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (c + e < a.c.d) dst[e] = round_to<T>(y[e]);
    }
  }
  if (slice == 0 && tid < rows) {
    const float l2 = s_l[tid] != 0.f ? s_m[tid] + log2f(s_l[tid]) : -INFINITY;
    if (a.lse) a.lse[(int64_t)b * a.hq + row0 + tid] = l2 * kLn2F;
    if (a.scores) a.lse2[(int64_t)b * a.hq + row0 + tid] = l2;
  }
  collect();
}


}  // namespace
}  // namespace sage
