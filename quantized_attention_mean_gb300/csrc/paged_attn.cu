// Attention of one new token per sequence over a paged key-value cache (sage_paged_attn).
//
//   t_j = sm_scale q.k_j, capped to cap tanh(t_j / cap), less slope |pos_q - pos_j|
//   out = sum_j softmax(t)_j v_j over the sequence's held tokens, lse = ln sum_j exp t_j
//
// Up to 16 query heads per key/value head every held K and V row is read once, so DRAM bounds it: a ragged batch of 32 sequences
// of up to 32K tokens (8 heads, head_dim 128) takes 280-284 us, 90% of what a copy's rate (6.8 TB/s) allows; two contexts of
// 50-60K tokens with their weights 175-178 us, 83%; a single short sequence 7.5 us in a graph, the latency of the chain length, page,
// row. The query heads of one key/value head are the rows of m16n8k16 products, in blocks of 16: a tcgen05 tile would have
// 128 rows, of which a decode step fills the same few, and the tensor work here is a small part of what the memory time
// allows. Each further block is an item of its own and reads the rows again, mostly from L2 where they fit: 8 sequences of 32K
// tokens, one key/value head, 8 query heads 35 us, 16 39, 32 51, 64 87.
//
// Split: the (sequence, head, key tile) items of the whole batch form one line, cut into equal
// ranges, one per CTA, so the load is even whatever the lengths (which only the device knows). Each
// warp takes 16 or 32 keys of a tile through its own ring of stages and keeps its own running maximum, sum
// and accumulator; no barrier runs inside a range. At a (sequence, head)'s last tile in a range the
// warps are merged in a fixed order; a result that lies in one range is written out, others go to
// the workspace and the join kernel sums them in the order of the ranges, so results do not depend
// on timing.
//
// Loads: pages of whole 8-row blocks come by TMA, a box of rows per lane, which costs the warp next to no
// instructions (16-byte cp.async per lane took 835 instructions per warp and tile and stalled at 4.6
// TB/s); tokens that are not there are boxes outside of the tensor and arrive as zeros. Other
// page sizes use cp.async, rows that no 16-byte load fits plain loads.
#include <cmath>
#include <cstring>

#include "../../include/sageattn.h"
#include "launch.h"
#include "paged.cuh"
#include "sm103_ptx.cuh"

namespace sage {
namespace {

constexpr int kWarps = 4;
constexpr int kCtas = 304;                 // two resident CTAs per SM
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
  int mass4;                // see mass_kernel
  int slices;               // CTAs of the join per (row block of a head, sequence)
  // workspace
  int* err;                 // status word, or null (no workspace: the clusters' form without mass)
  int* cta_err;             // [kCtas]
  float* part_o;            // [kCtas][2][kRows][dp]
  float* part_ml;           // [kCtas][2][kRows][2]
  float* lse2;              // [batch, hq], base 2 (with mass)
  float* scores;            // [batch, hq, score_pitch], base 2 (with mass) or null
  int64_t score_pitch;
};

template <int DP>
struct DecodeCfg {
  static constexpr int kStages = 3;
  static constexpr int kKeys = DP == 128 ? 16 : 32;           // keys per warp and tile (8 KB of K and V)
  static constexpr int kTile = kWarps * kKeys;                // keys per tile
  static constexpr int kChunks = DP / 64;                     // blocks of 64 channels, rows of 128 bytes
  static constexpr int kChunkBytes = kKeys * 128;
  static constexpr int kTileBytes = kChunks * kChunkBytes;    // K or V of one warp's tile
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kWarpBytes = kStages * kStageBytes;
  static constexpr int kOffMerge = kWarps * kWarpBytes;       // two warps' accumulators, 64 channels at a time
  static constexpr int kOffMl = kOffMerge + 2 * kRows * 64 * 4;
  static constexpr int kOffBar = kOffMl + kWarps * kRows * 2 * 4;
  static constexpr int kSmem = kOffBar + kWarps * kStages * 8;
};

// Tiles of a sequence of n tokens.
template <int DP>
__device__ __forceinline__ int tiles_of(int n) {
  return (n + DecodeCfg<DP>::kTile - 1) / DecodeCfg<DP>::kTile;
}

// The items (sequence, head, tile) of sequences [b0, b0 + blockDim): this thread's count, the sum before it and the
// sum of all. Lengths that are out of range count as 0 and set `bad`.
struct Scan {
  long long n, before, all;
};
template <int DP>
__device__ __forceinline__ Scan scan_items(const DecodeArgs& a, int heads, int b0, bool& bad) {
  __shared__ long long s_sum[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const int b = b0 + threadIdx.x;
  Scan r{0, 0, 0};
  if (b < a.c.batch) {
    const int len = checked_len(a.c, b, a.max_len);
    if (len < 0) bad = true;
    r.n = (long long)tiles_of<DP>(max(len, 0)) * heads;
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
__device__ __forceinline__ int ctas_of(long long total) {
  const long long g = (total + kMinTiles - 1) / kMinTiles;
  return (int)(g < kCtas ? g : kCtas);
}
__device__ __forceinline__ long long first_item(long long total, int ctas, int i) {
  return total * i / ctas;
}

// One place on the line of items.
struct Cursor {
  int b, h, tile, tiles, len;  // h: head * row_blocks + row block
};
template <int DP>
__device__ __forceinline__ void next_item(const DecodeArgs& a, int heads, Cursor& u) {
  if (++u.tile < u.tiles) return;
  u.tile = 0;
  if (++u.h < heads) return;
  u.h = 0;
  do {
    ++u.b;
    u.len = u.b < a.c.batch ? max(checked_len(a.c, u.b, a.max_len), 0) : 0;
  } while (u.b < a.c.batch && u.len == 0);
  u.tiles = tiles_of<DP>(u.len);
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

// The keys of an item that belong to this warp into one stage: K, then V, per 64 channels rows of 128
// bytes whose 16-byte unit c lies at c ^ (row & 7). Tokens that are not there and channels past d
// become zero. `page`, `slot`: TMA: of this lane's box (K or V by bit 0, channels by bit 1 at head_dim 128, rows by the
// rest); otherwise of row (lane mod the keys).
template <typename T, int DP>
__device__ __forceinline__ void load_stage(const DecodeArgs& a, const CUtensorMap* tmK, const CUtensorMap* tmV, int h,
                                           int page, int slot, uint8_t* stage, uint32_t bar) {
  using C = DecodeCfg<DP>;
  const int lane = threadIdx.x & 31;
  const uint32_t base = smem_u32(stage);
  if (a.load == kLoadTma) {
    if (lane == 0)
      asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(C::kStageBytes) : "memory");
    const int kv = lane & 1, chunk = C::kChunks == 2 ? (lane >> 1) & 1 : 0, rows = (lane >> C::kChunks) * a.box_rows;
    if (rows < C::kKeys)
      tma_box(base + kv * C::kTileBytes + chunk * C::kChunkBytes + rows * 128, kv ? tmV : tmK, bar, chunk * 64, slot, h,
              page >= 0 ? page : a.c.num_pages);
    return;
  }
  const T* none = reinterpret_cast<const T*>(reinterpret_cast<uintptr_t>(a.q) & ~static_cast<uintptr_t>(15));  // nothing is read from it
  const T* kb = static_cast<const T*>(a.c.k) + h * a.c.k_sh;
  const T* vb = static_cast<const T*>(a.c.v) + h * a.c.v_sh;
  constexpr int kUnits = DP / 8, kRowsPer = 32 / kUnits;  // rows that one pass of the warp covers
  const int c = lane % kUnits;
#pragma unroll 2
  for (int i = 0; i < C::kKeys / kRowsPer; ++i) {
    const int r = i * kRowsPer + lane / kUnits;
    const int pg = __shfl_sync(0xffffffffu, page, r), sl = __shfl_sync(0xffffffffu, slot, r);
    const bool in = pg >= 0 && c * 8 < a.c.d;
    const int off = (c >> 3) * C::kChunkBytes + r * 128 + (((c & 7) ^ (r & 7)) << 4);
    const T* ks = in ? kb + pg * a.c.k_sp + sl * a.c.k_st + c * 8 : none;
    const T* vs = in ? vb + pg * a.c.v_sp + sl * a.c.v_st + c * 8 : none;
    if (a.load == kLoadVec) {
      cp_async16(base + off, ks, in ? 16 : 0);
      cp_async16(base + C::kTileBytes + off, vs, in ? 16 : 0);
    } else {
      T* kd = reinterpret_cast<T*>(stage + off);
      T* vd = reinterpret_cast<T*>(stage + C::kTileBytes + off);
#pragma unroll 1
      for (int e = 0; e < 8; ++e) {
        const bool ok = in && c * 8 + e < a.c.d;
        kd[e] = ok ? ks[e] : T(0.0f);
        vd[e] = ok ? vs[e] : T(0.0f);
      }
    }
  }
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

// Rows r0 and r0 + 8 of a finished (sequence, head) from one warp's accumulators.
template <typename T, int DP>
__device__ __forceinline__ void write_rows(const DecodeArgs& a, int b, int row0, int rows,
                                           const float (&o)[DP / 8][4], float m0, float m1, float l0, float l1) {
  const int lane = threadIdx.x & 31, cq = (lane & 3) * 2;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int r = (lane >> 2) + half * 8;
    if (r >= rows) continue;
    const float m = half ? m1 : m0, l = half ? l1 : l0;
    const float inv = l != 0.f ? 1.0f / l : 0.f;
    T* dst = static_cast<T*>(a.o) + b * a.o_sb + (row0 + r) * a.o_sh;
#pragma unroll
    for (int n = 0; n < DP / 8; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (n * 8 + cq + e < a.c.d) dst[n * 8 + cq + e] = round_to<T>(o[n][2 * half + e] * inv);
    if ((lane & 3) == 0) {
      const float l2 = l != 0.f ? m + log2f(l) : -INFINITY;
      if (a.lse) a.lse[(int64_t)b * a.hq + row0 + r] = l2 * kLn2F;
      if (a.scores) a.lse2[(int64_t)b * a.hq + row0 + r] = l2;
    }
  }
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

// The kernel of both forms. CLUSTER: grid (kRanks x row blocks of heads, batch), each CTA of a cluster takes its
// share of one sequence's tiles; otherwise kCtas ranges of the line.
template <typename T, int DP, bool CLUSTER>
__global__ void __launch_bounds__(kWarps * 32, 2)
    decode_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const DecodeArgs a) {
  using C = DecodeCfg<DP>;
  constexpr int S = C::kStages, KS = DP / 16, NT = DP / 8, NK = C::kKeys / 8;
  // fp16 weights are held at up to 2^(7 + 8): 7 bits more before the smallest lose bits
  constexpr float kHead = std::is_same<T, __half>::value ? 7.0f : 0.f;
  extern __shared__ __align__(1024) uint8_t sm[];
  __shared__ int s_err[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int heads = a.c.hkv * a.row_blocks;
  uint8_t* const ring = sm + warp * C::kWarpBytes;
  float* const merge = reinterpret_cast<float*>(sm + C::kOffMerge);
  float* const ml = reinterpret_cast<float*>(sm + C::kOffMl);
  const uint32_t bars = smem_u32(sm + C::kOffBar) + warp * S * 8;
  if (lane < S) asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(bars + lane * 8) : "memory");
  fence_mbar_init();
  if (a.load == kLoadTma && lane == 0) {
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  pdl_wait();
  const int me = blockIdx.x;
  int err = 0;
  long long left = 0;
  Cursor cu{a.c.batch, 0, 0, 1, 0};
  __shared__ long long s_base;
  __shared__ int s_b;
  if constexpr (CLUSTER) {
    const int rank = me % kRanks;
    cu.b = blockIdx.y;
    cu.h = me / kRanks;
    cu.len = max(checked_len(a.c, cu.b, a.max_len), 0);
    cu.tiles = tiles_of<DP>(cu.len);
    cu.tile = cu.tiles * rank / kRanks;
    left = cu.tiles * (rank + 1) / kRanks - cu.tile;
  } else {
    // this CTA's range of the line: the total, then the sequence that its first item lies in
    bool bad = false;
    if (threadIdx.x == 0) { s_b = a.c.batch; s_base = 0; }
    Scan sc = scan_items<DP>(a, heads, 0, bad);
    long long total = sc.all;
    for (int b0 = blockDim.x; b0 < a.c.batch; b0 += blockDim.x) total += scan_items<DP>(a, heads, b0, bad).all;
    const int ctas = total > 0 ? ctas_of(total) : 0;
    long long i0 = 0;
    if (me < ctas) {
      i0 = first_item(total, ctas, me);
      left = first_item(total, ctas, me + 1) - i0;
      long long base = 0;
      for (int b0 = 0;;) {
        const long long lo = base + sc.before;
        if (sc.n > 0 && i0 >= lo && i0 < lo + sc.n) { s_b = b0 + threadIdx.x; s_base = lo; }
        base += sc.all;
        b0 += blockDim.x;
        if (base > i0 || b0 >= a.c.batch) break;
        sc = scan_items<DP>(a, heads, b0, bad);
      }
    }
    __syncthreads();
    err = bad ? kDevSeqlens : 0;
    if (left > 0) {
      cu.b = s_b;
      cu.len = checked_len(a.c, cu.b, a.max_len);
      cu.tiles = tiles_of<DP>(cu.len);
      const long long in = i0 - s_base;
      cu.h = (int)(in / cu.tiles);
      cu.tile = (int)(in - (long long)cu.h * cu.tiles);
    }
  }
  pdl_trigger();

  if constexpr (CLUSTER) {
    // the status word has one writer (but for a wait that runs out, two seconds from now): the first
    // CTA looks at the lengths and pages of all sequences
    if (a.err && me == 0 && blockIdx.y == 0) {
      int e = 0;
      for (int b = 0; b < a.c.batch; ++b) {
        const int len = checked_len(a.c, b, a.max_len);
        if (len < 0) e = max(e, (int)kDevSeqlens);
        for (int i = threadIdx.x; i < (len + a.c.page_size - 1) / a.c.page_size; i += kWarps * 32) {
          const int pg = __ldg(&a.c.table[b * a.c.table_stride + i]);
          if (pg < 0 || pg >= a.c.num_pages) e = max(e, kDevPage);
        }
      }
      e = __reduce_max_sync(0xffffffffu, e);
      if (lane == 0) s_err[warp] = e;
      __syncthreads();
      if (threadIdx.x == 0) *a.err = max(max(s_err[0], s_err[1]), max(s_err[2], s_err[3]));
    }
  }
  // ---- fill the ring: S - 1 stages in flight, the page of the stage after them already read
  Cursor ld = cu;
  long long to_load = left;
  int page, slot;
  const int my_row = a.load == kLoadTma ? (lane >> C::kChunks) * a.box_rows : lane & (C::kKeys - 1);
  auto next_page = [&]() {
    const int key = ld.tile * C::kTile + warp * C::kKeys + my_row;
    find_page(a, ld.b, key, to_load > 0 && my_row < C::kKeys && key < ld.len, page, slot, err);
  };
  bool dead = false;  // a wait has run out: nothing more is loaded
  auto load_next = [&](int st) {
    if (to_load > 0 && !dead) {
      load_stage<T, DP>(a, &tmK, &tmV, ld.h / a.row_blocks, page, slot, ring + st * C::kStageBytes, bars + st * 8);
      next_item<DP>(a, heads, ld);
      --to_load;
      next_page();
    }
    if (a.load != kLoadTma) cp_async_commit();
  };
  __syncwarp();
  next_page();
#pragma unroll 1
  for (int st = 0; st < S - 1; ++st) load_next(st);

  float o[NT][4], m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
  uint32_t qf[KS][4];
  float sl0 = 0.f, sl1 = 0.f;
  int qpos = 0, rows = 0, row0 = 0, tile0 = 0, pieces = 0;
  bool fresh = true;
  if constexpr (CLUSTER) {
    const int rb = cu.h % a.row_blocks;
    row0 = cu.h / a.row_blocks * a.group + rb * kRows;
    rows = min(kRows, a.group - rb * kRows);
  }
  const float scale2 = a.sm_scale * kLog2eF;
  const float cap_in = a.cap > 0.f ? a.sm_scale / a.cap : 0.f, cap_out = a.cap * kLog2eF;
  int stage = 0;
  uint32_t parity = 0;
  const int r0 = lane >> 2, cq = (lane & 3) * 2;

#pragma unroll 1
  for (; left > 0; --left) {
    if (fresh) {
      // a new (sequence, head): its query rows as the A operand, its statistics
      fresh = false;
      tile0 = cu.tile;
      const int h = cu.h / a.row_blocks, rb = cu.h - h * a.row_blocks;
      row0 = h * a.group + rb * kRows;
      rows = min(kRows, a.group - rb * kRows);
      const T* qb = static_cast<const T*>(a.q) + cu.b * a.q_sb;
      auto at = [&](int r, int c) {
        return r < rows && c < a.c.d ? qb[(row0 + r) * a.q_sh + c] : T(0.0f);
      };
      auto two = [&](int r, int c) {
        T x[2] = {at(r, c), at(r, c + 1)};
        return *reinterpret_cast<const uint32_t*>(x);
      };
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        qf[k][0] = two(r0, k * 16 + cq);
        qf[k][1] = two(r0 + 8, k * 16 + cq);
        qf[k][2] = two(r0, k * 16 + 8 + cq);
        qf[k][3] = two(r0 + 8, k * 16 + 8 + cq);
      }
      sl0 = sl1 = 0.f;
      if (a.slopes) {
        if (r0 < rows) sl0 = __ldg(&a.slopes[row0 + r0]) * kLog2eF;
        if (r0 + 8 < rows) sl1 = __ldg(&a.slopes[row0 + r0 + 8]) * kLog2eF;
      }
      qpos = a.q_pos ? __ldg(&a.q_pos[cu.b]) : cu.len - 1;
#pragma unroll
      for (int n = 0; n < NT; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
      m0 = m1 = -INFINITY;
      l0 = l1 = 0.f;
    }
    // the stage after the ones in flight goes where the previous item was
    __syncwarp();
    load_next(stage == 0 ? S - 1 : stage - 1);
    const int key0 = cu.tile * C::kTile + warp * C::kKeys;
    uint8_t* const here = ring + stage * C::kStageBytes;
    if (a.load == kLoadTma) {
      if (!dead && !__all_sync(0xffffffffu, wait_stage(bars + stage * 8, parity))) {
        dead = true;
        err = kDevTimeout;
        // what is in flight lands (or runs out of time) before the shared memory goes away
        for (int k = 0; k < (int)(left - to_load); ++k) {
          const int st = stage + k;
          wait_stage(bars + (st % S) * 8, parity ^ (st >= S ? 1u : 0u));
        }
      }
      if (!dead && key0 < cu.len && key0 + C::kKeys > cu.len) {
        // slots behind the last token may hold anything: as V rows they become zero (their scores are masked)
        for (int i = lane; i < (key0 + C::kKeys - cu.len) * C::kChunks * 8; i += 32) {
          const int r = cu.len - key0 + i / (C::kChunks * 8), u = i % (C::kChunks * 8);
          *reinterpret_cast<uint4*>(here + C::kTileBytes + (u >> 3) * C::kChunkBytes + r * 128 + (u & 7) * 16) =
              make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
      }
    } else {
      cp_async_wait<S - 1>();
    }
    __syncwarp();
    if (key0 < cu.len) {
      const bool upper = rows > 8;  // rows r0 + 8 are in use
      const uint32_t kb = smem_u32(here), vb = kb + C::kTileBytes;
      // S = Q K^T, 16 keys at a time: lanes 0-7 / 8-15 address keys 0-7 at channels +0 / +8, 16-23 / 24-31 keys
      // 8-15; two accumulators per 8 keys, so that no chain is longer than half the channels
      float s[NK][4], s2[NK][4];
#pragma unroll
      for (int n = 0; n < NK; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] = s2[n][e] = 0.f;
      {
        const int r = (lane & 7) + ((lane >> 4) << 3), odd = (lane >> 3) & 1;
        const uint32_t row = kb + r * 128;
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int n = 0; n < NK; n += 2) {
            uint32_t b[4];
            ldsm4(row + n * 1024 + (k >> 2) * C::kChunkBytes + (((((2 * k) & 7) + odd) ^ (r & 7)) << 4), b);
            mma16816<T>(k & 1 ? s2[n] : s[n], qf[k], b[0], b[1]);
            mma16816<T>(k & 1 ? s2[n + 1] : s[n + 1], qf[k], b[2], b[3]);
          }
      }
#pragma unroll
      for (int n = 0; n < NK; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] += s2[n][e];
      // scores in base 2; lane holds keys 8 n + cq, + 1 of rows r0 (s[n][0..1]) and r0 + 8
      if (a.cap > 0.f) {
#pragma unroll
        for (int n = 0; n < NK; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (e < 2 || upper) s[n][e] = tanhf(s[n][e] * cap_in) * cap_out;
      } else {
#pragma unroll
        for (int n = 0; n < NK; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][e] *= scale2;
      }
      if (a.slopes && !a.c.pos) {
        const float d0 = (float)((long long)qpos - (key0 + cq));  // exact below 2^24
#pragma unroll
        for (int n = 0; n < NK; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float dist = fabsf(d0 - (float)(n * 8 + e));
            s[n][e] = fmaf(-sl0, dist, s[n][e]);
            s[n][2 + e] = fmaf(-sl1, dist, s[n][2 + e]);
          }
      } else if (a.slopes) {
#pragma unroll 1
        for (int n = 0; n < NK; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int key = key0 + n * 8 + cq + e;
            int pg, sl, none = 0;
            find_page(a, cu.b, key, key < cu.len, pg, sl, none);
            const int kp = pg >= 0 ? __ldg(&a.c.pos[plane_at(a.c, pg, cu.h / a.row_blocks, sl)]) : 0;
            const float dist = fabsf((float)((long long)qpos - kp));
#pragma unroll
            for (int u = 0; u < NK; ++u)
              if (u == n) {
                s[u][e] = fmaf(-sl0, dist, s[u][e]);
                s[u][2 + e] = fmaf(-sl1, dist, s[u][2 + e]);
              }
          }
      }
      if (key0 + C::kKeys > cu.len) {
#pragma unroll
        for (int n = 0; n < NK; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (key0 + n * 8 + cq + (e & 1) >= cu.len) s[n][e] = -INFINITY;
      }
      if (a.scores) {
        // (the pitch is a multiple of the tile, so pairs are aligned and whole tiles fit)
        float* dst = a.scores + ((int64_t)cu.b * a.hq + row0 + r0) * a.score_pitch + key0 + cq;
        if (r0 < rows) {
#pragma unroll
          for (int n = 0; n < NK; ++n) *reinterpret_cast<float2*>(dst + n * 8) = make_float2(s[n][0], s[n][1]);
        }
        if (r0 + 8 < rows) {
#pragma unroll
          for (int n = 0; n < NK; ++n)
            *reinterpret_cast<float2*>(dst + 8 * a.score_pitch + n * 8) = make_float2(s[n][2], s[n][3]);
        }
      }
      // the frame of a row (its four lanes agree) lies kHead below the maximum that set it, and is
      // kept unless that grew by more than 8: the sums and O are rescaled rarely
      float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
      for (int n = 0; n < NK; ++n) {
        x0 = max3(x0, s[n][0], s[n][1]);
        x1 = max3(x1, s[n][2], s[n][3]);
      }
#pragma unroll
      for (int w = 1; w < 4; w <<= 1) {
        x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, w));
        if (upper) x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, w));
      }
      x0 -= kHead;
      x1 -= kHead;
      const bool g0 = x0 > m0 + 8.0f || (m0 == -INFINITY && x0 > -INFINITY);
      const bool g1 = x1 > m1 + 8.0f || (m1 == -INFINITY && x1 > -INFINITY);
      if (__any_sync(0xffffffffu, g0 || g1)) {
        const float f0 = g0 ? ex2_approx(m0 - x0) : 1.0f, f1 = g1 ? ex2_approx(m1 - x1) : 1.0f;
        l0 *= f0;
        l1 *= f1;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          o[n][0] *= f0; o[n][1] *= f0;
          o[n][2] *= f1; o[n][3] *= f1;
        }
        m0 = g0 ? x0 : m0;
        m1 = g1 ? x1 : m1;
      }
      const float u0 = m0 == -INFINITY ? 0.f : m0, u1 = m1 == -INFINITY ? 0.f : m1;
#pragma unroll
      for (int n = 0; n < NK; ++n) {
        s[n][0] = ex2_approx(s[n][0] - u0);
        s[n][1] = ex2_approx(s[n][1] - u0);
        s[n][2] = upper ? ex2_approx(s[n][2] - u1) : 0.f;
        s[n][3] = upper ? ex2_approx(s[n][3] - u1) : 0.f;
        l0 += s[n][0] + s[n][1];
        l1 += s[n][2] + s[n][3];
      }
      // P in the operands' 16-bit type (the one rounding of the weights; their sum stays in
      // 32 bits), which is already the A operand's layout; O += P V, 16 keys at a time
#pragma unroll
      for (int g = 0; g < NK; g += 2) {
        const uint32_t p[4] = {pack2<T>(s[g][0], s[g][1]), pack2<T>(s[g][2], s[g][3]),
                               pack2<T>(s[g + 1][0], s[g + 1][1]), pack2<T>(s[g + 1][2], s[g + 1][3])};
        const int r = (lane & 7) + (((lane >> 3) & 1) << 3), hi = lane >> 4;  // keys 0-7 / 8-15
        const uint32_t row = vb + g * 1024 + r * 128;
#pragma unroll
        for (int n = 0; n < NT; n += 2) {
          uint32_t b[4];
          ldsm4t(row + (n >> 3) * C::kChunkBytes + ((((n & 7) + hi) ^ (r & 7)) << 4), b);
          mma16816<T>(o[n], p, b[0], b[1]);
          mma16816<T>(o[n + 1], p, b[2], b[3]);
        }
      }
    }
    if (stage + 1 == S) {
      stage = 0;
      parity ^= 1;
    } else {
      ++stage;
    }
    const bool seg_end = !CLUSTER && (cu.tile + 1 == cu.tiles || left == 1);
    if (seg_end) {
      // ---- merge the warps: sums of a row over its four lanes, then over the warps
#pragma unroll
      for (int w = 1; w < 4; w <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, w);
        l1 += __shfl_xor_sync(0xffffffffu, l1, w);
      }
      if ((lane & 3) == 0) {
        ml[(warp * kRows + r0) * 2] = m0;
        ml[(warp * kRows + r0) * 2 + 1] = l0;
        ml[(warp * kRows + r0 + 8) * 2] = m1;
        ml[(warp * kRows + r0 + 8) * 2 + 1] = l1;
      }
      __syncthreads();
      float M0 = -INFINITY, M1 = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        M0 = fmaxf(M0, ml[(w * kRows + r0) * 2]);
        M1 = fmaxf(M1, ml[(w * kRows + r0 + 8) * 2]);
      }
      const float U0 = M0 == -INFINITY ? 0.f : M0, U1 = M1 == -INFINITY ? 0.f : M1;
      float L0 = 0.f, L1 = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        L0 += ml[(w * kRows + r0) * 2 + 1] * ex2_approx(ml[(w * kRows + r0) * 2] - U0);
        L1 += ml[(w * kRows + r0 + 8) * 2 + 1] * ex2_approx(ml[(w * kRows + r0 + 8) * 2] - U1);
      }
      const float f0 = ex2_approx(m0 - U0), f1 = ex2_approx(m1 - U1);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        o[n][0] *= f0; o[n][1] *= f0;
        o[n][2] *= f1; o[n][3] *= f1;
      }
      // pairs (0, 2) and (1, 3), then (0, 1)
#pragma unroll
      for (int c = 0; c < NT; c += 8)
#pragma unroll
        for (int step = 2; step >= 1; step >>= 1) {
          if (warp >= step && warp < 2 * step) {
            float* dst = merge + (warp - step) * kRows * 64 + r0 * 64 + cq;
#pragma unroll
            for (int n = 0; n < 8; ++n) {
              *reinterpret_cast<float2*>(dst + n * 8) = make_float2(o[c + n][0], o[c + n][1]);
              if (rows > 8) *reinterpret_cast<float2*>(dst + 8 * 64 + n * 8) = make_float2(o[c + n][2], o[c + n][3]);
            }
          }
          __syncthreads();
          if (warp < step) {
            const float* src = merge + warp * kRows * 64 + r0 * 64 + cq;
#pragma unroll
            for (int n = 0; n < 8; ++n) {
              const float2 x = *reinterpret_cast<const float2*>(src + n * 8);
              o[c + n][0] += x.x; o[c + n][1] += x.y;
              if (rows > 8) {
                const float2 y = *reinterpret_cast<const float2*>(src + 8 * 64 + n * 8);
                o[c + n][2] += y.x; o[c + n][3] += y.y;
              }
            }
          }
          __syncthreads();
        }
      if (warp == 0) {
        // the whole (sequence, head) in this range: the result; a part of it: to the workspace
        const bool whole = tile0 == 0 && cu.tile + 1 == cu.tiles;
        if (whole) {
          write_rows<T, DP>(a, cu.b, row0, rows, o, M0, M1, L0, L1);
        } else {
          const int64_t at = ((int64_t)me * 2 + (pieces > 0)) * kRows;
          float* po = a.part_o + at * DP;
          float* pm = a.part_ml + at * 2;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int r = r0 + half * 8;
            if (r < rows) {
#pragma unroll
              for (int n = 0; n < NT; ++n)
                *reinterpret_cast<float2*>(po + r * DP + n * 8 + cq) =
                    make_float2(o[n][2 * half], o[n][2 * half + 1]);
              if ((lane & 3) == 0)
                *reinterpret_cast<float2*>(pm + r * 2) = make_float2(half ? M1 : M0, half ? L1 : L0);
            }
          }
        }
      }
      ++pieces;
      fresh = true;
    }
    next_item<DP>(a, heads, cu);
  }
  if constexpr (CLUSTER) {
    // every warp's accumulator into its own ring, its statistics beside; then each thread of the
    // cluster sums one group of four channels of a row over all warps of all ranks, in their order
    const int rank = me % kRanks;
#pragma unroll
    for (int w = 1; w < 4; w <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, w);
      l1 += __shfl_xor_sync(0xffffffffu, l1, w);
    }
    __syncwarp();
    float* const mine = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int r = r0 + half * 8;
      if (!fresh && r < rows) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
          *reinterpret_cast<float2*>(mine + r * DP + n * 8 + cq) = make_float2(o[n][2 * half], o[n][2 * half + 1]);
      }
      if ((lane & 3) == 0)
        *reinterpret_cast<float2*>(&ml[(warp * kRows + r) * 2]) =
            fresh ? make_float2(-INFINITY, 0.f) : make_float2(half ? m1 : m0, half ? l1 : l0);
    }
    if (dead && a.err) record_error(a.err, kDevTimeout);
    cluster_sync();
    const int cell = rank * kWarps * 32 + threadIdx.x, r = cell / (DP / 4), c = (cell - r * (DP / 4)) * 4;
    if (r < rows) {
      const uint32_t ml_at = smem_u32(ml + r * 2), o_at = smem_u32(sm) + (r * DP + c) * 4;
      float2 st[kRanks * kWarps];
#pragma unroll
      for (int p = 0; p < kRanks * kWarps; ++p) st[p] = ld_rank2(of_rank(ml_at + (p % kWarps) * kRows * 8, p / kWarps));
      float m = -INFINITY, l = 0.f;
#pragma unroll
      for (int p = 0; p < kRanks * kWarps; ++p) m = fmaxf(m, st[p].x);
      const float u = m == -INFINITY ? 0.f : m;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int p = 0; p < kRanks * kWarps; ++p) {
        const float w = ex2_approx(st[p].x - u);
        l = fmaf(st[p].y, w, l);
        if (st[p].y != 0.f) {  // (a warp without keys wrote no accumulator)
          const float4 x = ld_rank4(of_rank(o_at + (p % kWarps) * C::kWarpBytes, p / kWarps));
          acc.x = fmaf(w, x.x, acc.x); acc.y = fmaf(w, x.y, acc.y);
          acc.z = fmaf(w, x.z, acc.z); acc.w = fmaf(w, x.w, acc.w);
        }
      }
      const float inv = l != 0.f ? 1.0f / l : 0.f;
      const float y[4] = {acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv};
      T* dst = static_cast<T*>(a.o) + (int64_t)blockIdx.y * a.o_sb + (row0 + r) * a.o_sh + c;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (c + e < a.c.d) dst[e] = round_to<T>(y[e]);
      if (c == 0) {
        const float l2 = l != 0.f ? m + log2f(l) : -INFINITY;
        const int64_t at = (int64_t)blockIdx.y * a.hq + row0 + r;
        if (a.lse) a.lse[at] = l2 * kLn2F;
        if (a.scores) a.lse2[at] = l2;
      }
    }
    cluster_sync();  // no CTA's shared memory goes away while it is read
    return;
  }
  // this CTA's error, collected by the join kernel (no word to clear before the call)
  const int we = __reduce_max_sync(0xffffffffu, err);
  if (lane == 0) s_err[warp] = we;
  __syncthreads();
  if (threadIdx.x == 0) {
    int e = 0;
    for (int w = 0; w < kWarps; ++w) e = max(e, s_err[w]);
    a.cta_err[me] = e;
  }
}

// ------------------------------------------------------------------------------------- join
// One CTA per (row block of a head, sequence), or per 32 of its channels: the results that lie in several ranges summed in
// the order of the ranges; sequences that hold nothing get 0 and -inf. CTA (0, 0) also collects the status.
constexpr int kJoinThreads = 256;

template <typename T, int DP>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const DecodeArgs a) {
  __shared__ float s_w[kCtas][kRows];       // weight of each range's piece
  __shared__ int s_at[kCtas];               // and where it lies
  __shared__ float s_m[kRows], s_l[kRows];
  __shared__ __align__(16) float s_acc[kJoinThreads * 4];
  __shared__ long long s_before[kJoinThreads / 32], s_all[kJoinThreads / 32];
  const int heads = a.c.hkv * a.row_blocks;
  const int hb = blockIdx.x / a.slices, slice = blockIdx.x - hb * a.slices;
  const int b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0 && b == 0) {
    int e = 0;
    for (int i = tid; i < kCtas; i += kJoinThreads) e = max(e, a.cta_err[i]);
    e = __reduce_max_sync(0xffffffffu, e);
    if (lane == 0) s_all[warp] = e;
    __syncthreads();
    if (tid == 0) {
      for (int w = 0; w < kJoinThreads / 32; ++w) e = max(e, (int)s_all[w]);
      *a.err = e;
    }
    __syncthreads();
  }
  // items before this sequence, and in all
  long long before = 0, all = 0;
  for (int i = tid; i < a.c.batch; i += kJoinThreads) {
    const long long n = (long long)tiles_of<DP>(max(checked_len(a.c, i, a.max_len), 0)) * heads;
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
    if (slice > 0) return;
    for (int i = tid; i < rows * a.c.d; i += kJoinThreads) {
      const int r = i / a.c.d, c = i - r * a.c.d;
      static_cast<T*>(a.o)[b * a.o_sb + (row0 + r) * a.o_sh + c] = T(0.0f);
    }
    if (a.lse && tid < rows) a.lse[(int64_t)b * a.hq + row0 + tid] = -INFINITY;
    return;
  }
  const long long t0 = before + (long long)hb * tiles_of<DP>(len), t1 = t0 + tiles_of<DP>(len);
  const int ctas = ctas_of(all);
  // the ranges that hold t0 and t1 - 1: range i is [all i / ctas, all (i + 1) / ctas)
  auto range_of = [&](long long t) { return (int)(((t + 1) * ctas - 1) / all); };
  const int c0 = range_of(t0), c1 = range_of(t1 - 1);
  if (c0 == c1) return;  // written by its own range
  const int parts = c1 - c0 + 1;
  // a range's first piece is this one's unless it starts before it
  for (int p = tid; p < parts; p += kJoinThreads) s_at[p] = (c0 + p) * 2 + (first_item(all, ctas, c0 + p) < t0 ? 1 : 0);
  __syncthreads();
  // row statistics: one warp per row
  for (int r = warp; r < rows; r += kJoinThreads / 32) {
    float m = -INFINITY;
    for (int p = lane; p < parts; p += 32) m = fmaxf(m, a.part_ml[(s_at[p] * kRows + r) * 2]);
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
    const float u = m == -INFINITY ? 0.f : m;
    float l = 0.f;
    for (int p = lane; p < parts; p += 32) {
      const float2 x = *reinterpret_cast<const float2*>(a.part_ml + (s_at[p] * kRows + r) * 2);
      const float w = ex2_approx(x.x - u);
      s_w[p][r] = w;
      l += x.y * w;
    }
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) l += __shfl_xor_sync(0xffffffffu, l, w);
    if (lane == 0) { s_m[r] = m; s_l[r] = l; }
  }
  __syncthreads();
  // accumulators, four channels per thread; threads left over take every n-th piece
  const int groups = DP / 4 / a.slices, cells = rows * groups;  // groups of four channels
  const int sets = cells >= kJoinThreads ? 1 : kJoinThreads / cells;
  for (int base = 0; base < cells; base += kJoinThreads) {
    const int set = sets > 1 ? tid / cells : 0;
    const int cell = sets > 1 ? tid - set * cells : base + tid;
    const bool on = set < sets && cell < cells;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    const int r = on ? cell / groups : 0, c = (slice * groups + (on ? cell - r * groups : 0)) * 4;
    if (on) {
#pragma unroll 8
      for (int p = set; p < parts; p += sets) {
        const float4 x = *reinterpret_cast<const float4*>(a.part_o + ((int64_t)s_at[p] * kRows + r) * DP + c);
        const float w = s_w[p][r];
        acc.x = fmaf(w, x.x, acc.x); acc.y = fmaf(w, x.y, acc.y);
        acc.z = fmaf(w, x.z, acc.z); acc.w = fmaf(w, x.w, acc.w);
      }
    }
    if (sets > 1) {
      *reinterpret_cast<float4*>(&s_acc[tid * 4]) = acc;
      __syncthreads();
      if (tid < cells)
        for (int s = 1; s < sets; ++s) {
          const float4 x = *reinterpret_cast<const float4*>(&s_acc[(s * cells + tid) * 4]);
          acc.x += x.x; acc.y += x.y; acc.z += x.z; acc.w += x.w;
        }
    }
    if (on && set == 0) {
      const float inv = s_l[r] != 0.f ? 1.0f / s_l[r] : 0.f;
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
}

// --------------------------------------------------------------------------- accumulated weight
// mass += sum over the group's heads of 2^(t - lse2): the scores written by the decode kernel, four keys per
// thread. Added atomically, since two sequences may share a page; a page of one sequence gets one
// addition, whose result does not depend on any order. (`mass4`: four slots lie in one page and in one
// aligned 16 bytes of the plane.)
constexpr int kMassKeys = 4;
__global__ void __launch_bounds__(256) mass_kernel(const DecodeArgs a) {
  pdl_wait();
  const int b = blockIdx.z, h = blockIdx.y;
  const int len = max(checked_len(a.c, b, a.max_len), 0);
  const int key = (blockIdx.x * 256 + threadIdx.x) * kMassKeys;
  if (key >= len) return;
  const int64_t row = (int64_t)b * a.hq + h * a.group;
  const float* s = a.scores + row * a.score_pitch + key;  // (the pitch is a multiple of 128)
  float sum[kMassKeys] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int g = 0; g < a.group; ++g) {
    const float l2 = a.lse2[row + g];
    const float4 t = *reinterpret_cast<const float4*>(s + g * a.score_pitch);
    if (l2 != -INFINITY) {
      sum[0] += ex2_approx(t.x - l2);
      sum[1] += ex2_approx(t.y - l2);
      sum[2] += ex2_approx(t.z - l2);
      sum[3] += ex2_approx(t.w - l2);
    }
  }
  const int n = min(kMassKeys, len - key);
  int err = 0;
  if (a.mass4 && n == kMassKeys) {
    int page, slot;
    find_page(a, b, key, true, page, slot, err);
    if (page >= 0)
      asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(&a.c.mass[plane_at(a.c, page, h, slot)]),
                   "f"(sum[0]), "f"(sum[1]), "f"(sum[2]), "f"(sum[3])
                   : "memory");
    return;
  }
  for (int i = 0; i < n; ++i) {
    int page, slot;
    find_page(a, b, key + i, true, page, slot, err);
    if (page >= 0) atomicAdd(&a.c.mass[plane_at(a.c, page, h, slot)], sum[i]);
  }
}

// ------------------------------------------------------------------------------------- host
struct DecodeLayout {
  size_t err, part_o, part_ml, lse2, scores, total;
  int64_t pitch;
};
size_t up256(size_t x) { return (x + 255) / 256 * 256; }
// Few heads with short sequences: one launch of clusters whose CTAs all run at once, a tile or a few each, joined
// through distributed shared memory. Otherwise the line, which balances any lengths but takes a second launch
// to join. us in a graph, clusters and line, head_dim 128: 8 heads of 1000 tokens 7.4 and 11.0, of 4000 14.3 and 14.9,
// of 8000 23.5 and 17.4; 16 of 2000 11.1 and 13.2; 38 of 300 11.5 and 13.4, of 4000 29.2 and 22.1; 128 of 300 25.8 and 17.6.
bool clustered(int batch, int hkv, int row_blocks, int64_t max_len, int d) {
  const int tile = d <= 64 ? DecodeCfg<64>::kTile : DecodeCfg<128>::kTile;
  return (int64_t)hkv * row_blocks * batch * kRanks <= kCtas && max_len <= 8 * kRanks * tile;
}
bool decode_layout(int batch, int hq, int hkv, int64_t max_len, int d, bool mass, DecodeLayout* L) {
  if (batch < 0 || hq < 1 || hkv < 1 || hq % hkv || max_len < 0 || d < 1 || d > 128) return false;
  const int dp = d <= 64 ? 64 : 128;
  // status word; the line's ranges: their errors and their pieces
  const bool line = !clustered(batch, hkv, (hq / hkv + kRows - 1) / kRows, max_len, d);
  size_t o = 256 + (line ? up256(4 * kCtas) : 0);
  auto take = [&](size_t bytes) { const size_t at = o; o += up256(bytes); return at; };
  L->err = 256;
  L->part_o = take(line ? (size_t)kCtas * 2 * kRows * dp * 4 : 0);
  L->part_ml = take(line ? (size_t)kCtas * 2 * kRows * 2 * 4 : 0);
  L->pitch = (max_len + 127) / 128 * 128;  // whole tiles of either head_dim
  L->lse2 = take(mass ? (size_t)batch * hq * 4 : 0);
  L->scores = take(mass ? (size_t)batch * hq * L->pitch * 4 : 0);
  L->total = o;
  return true;
}

template <typename T, int DP>
cudaError_t launch_decode_t(const DecodeArgs& a, const CUtensorMap* maps, cudaStream_t st) {
  using C = DecodeCfg<DP>;
  const int heads = a.c.hkv * a.row_blocks;
  cudaError_t e;
  if (clustered(a.c.batch, a.c.hkv, a.row_blocks, a.max_len, a.c.d)) {
    static std::atomic<int> limits[64];
    e = raise_smem_limit(decode_kernel<T, DP, true>, C::kSmem, limits);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(heads * kRanks, a.c.batch);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kRanks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, decode_kernel<T, DP, true>, maps[0], maps[1], a);
  } else {
    static std::atomic<int> limits[64];
    e = raise_smem_limit(decode_kernel<T, DP, false>, C::kSmem, limits);
    if (e != cudaSuccess) return e;
    e = launch_pdl(decode_kernel<T, DP, false>, dim3(kCtas), dim3(kWarps * 32), C::kSmem, st, maps[0], maps[1], a);
    if (e != cudaSuccess) return e;
    e = launch_pdl(join_kernel<T, DP>, dim3(heads * a.slices, a.c.batch), dim3(kJoinThreads), 0, st, a);
  }
  if (e != cudaSuccess || !a.scores || a.max_len == 0) return e;
  return launch_pdl(mass_kernel, dim3((unsigned)(((int64_t)a.max_len + 256 * kMassKeys - 1) / (256 * kMassKeys)), a.c.hkv, a.c.batch), dim3(256), 0,
                    st, a);
}

}  // namespace
}  // namespace sage

using namespace sage;

extern "C" {

size_t sage_paged_attn_workspace_size(int batch, int heads_q, int heads_kv, int max_seqlen, int head_dim,
                                      int accumulate) {
  DecodeLayout L;
  return decode_layout(batch, heads_q, heads_kv, max_seqlen, head_dim, accumulate != 0, &L) ? L.total : 0;
}

int sage_paged_attn(const sage_packed* q, const sage_paged_cache* cache, const sage_packed* out, float* lse,
                    const float* slopes, const int32_t* q_positions, int batch, int heads_q, int heads_kv,
                    int max_seqlen, int head_dim, int dtype, int tensor_layout, float sm_scale, float softcap,
                    void* workspace, size_t workspace_bytes, void* stream) {
  if (!q || !cache || !out) return SAGE_ERR_INVALID_ARG;
  DecodeArgs a{};
  bool vec = false;
  int s = make_paged_view(cache, batch, heads_kv, head_dim, dtype, tensor_layout, &a.c, &vec);
  if (s != SAGE_OK) return s;
  if (heads_q < 1 || max_seqlen < 0 || batch > 65535 || !softcap_ok(softcap, sm_scale, head_dim))
    return SAGE_ERR_INVALID_ARG;
  if (heads_q % heads_kv) return SAGE_ERR_GQA;
  if (batch == 0) return SAGE_OK;
  if (!q->data || !out->data) return SAGE_ERR_INVALID_ARG;
  for (const sage_packed* t : {q, out})
    if (reinterpret_cast<uintptr_t>(t->data) % 2 || t->stride_token < 0 || t->stride_head < 0) return SAGE_ERR_STRIDE;
  for (const void* p : {(const void*)lse, (const void*)slopes, (const void*)q_positions})
    if (reinterpret_cast<uintptr_t>(p) % 4) return SAGE_ERR_INVALID_ARG;
  DecodeLayout L;
  if (!decode_layout(batch, heads_q, heads_kv, max_seqlen, head_dim, cache->mass != nullptr, &L))
    return SAGE_ERR_INVALID_ARG;
  // (the status word alone can do without)
  if (workspace ? reinterpret_cast<uintptr_t>(workspace) % 256 || workspace_bytes < L.total : L.total > SAGE_STATUS_BYTES)
    return SAGE_ERR_WORKSPACE;
  if (!sage_device_supported()) return SAGE_ERR_DEVICE;
  a.q = q->data; a.q_sb = q->stride_token; a.q_sh = q->stride_head;
  a.o = out->data; a.o_sb = out->stride_token; a.o_sh = out->stride_head;
  a.lse = lse;
  a.slopes = slopes;
  a.q_pos = q_positions;
  a.sm_scale = std::isnan(sm_scale) || sm_scale <= 0.f ? (float)(1.0 / std::sqrt((double)head_dim)) : sm_scale;
  a.cap = softcap;
  a.hq = heads_q;
  a.group = heads_q / heads_kv;
  a.row_blocks = (a.group + kRows - 1) / kRows;
  a.max_len = max_seqlen;
  // TMA: whole 16-byte rows, pages of whole 8-row blocks, no zero stride of a dimension that is walked
  const sage_paged_cache& pc = *cache;
  const int64_t len[3] = {pc.num_pages, tensor_layout == SAGE_HND ? heads_kv : pc.page_size,
                          tensor_layout == SAGE_HND ? pc.page_size : heads_kv};
  bool tma = vec && pc.page_size % 8 == 0;
  for (int i = 0; i < 3; ++i)
    tma = tma && (len[i] == 1 || (pc.k_stride[i] > 0 && pc.v_stride[i] > 0 && pc.k_stride[i] < (1LL << 38) &&
                                  pc.v_stride[i] < (1LL << 38))) && len[i] > 0;
  a.load = tma ? kLoadTma : vec ? kLoadVec : kLoadAny;
  const int keys = head_dim <= 64 ? DecodeCfg<64>::kKeys : DecodeCfg<128>::kKeys;
  a.box_rows = pc.page_size % keys == 0 ? keys : pc.page_size % 16 == 0 ? 16 : 8;
  a.page_shift = -1;
  for (int i = 0; i < 31; ++i)
    if (pc.page_size == 1 << i) a.page_shift = i;
  // the join by 32 channels where its CTAs would leave SMs idle (head_dim 128, us by slices and whole: 8 heads of 20000 tokens
  // 24.3 and 26.0, 16 of 2000 13.2 and 14.2, 38 of 20000 68.9 and 71.0; 64 of 20000 111.8 and 108.7, 256 of 2000 56.0 and 53.0;
  // head_dim 64 within 2%)
  a.slices = (int64_t)heads_kv * a.row_blocks * batch <= 38 ? (head_dim <= 64 ? 2 : 4) : 1;
  CUtensorMap maps[2];
  std::memset(maps, 0, sizeof(maps));
  if (tma) {
    auto map = [&](CUtensorMap* m, const void* base, int64_t sp, int64_t sh, int64_t st) {
      // (a stride that is never walked is given a legal value)
      return make_map4(m, dtype == SAGE_BF16, base, head_dim, pc.page_size, heads_kv, pc.num_pages, st * 2,
                       (heads_kv > 1 ? sh : 128) * 2, (pc.num_pages > 1 ? sp : 128) * 2, 64, a.box_rows);
    };
    if (!map(&maps[0], pc.k, a.c.k_sp, a.c.k_sh, a.c.k_st) || !map(&maps[1], pc.v, a.c.v_sp, a.c.v_sh, a.c.v_st))
      return note_cuda_failure(cudaErrorInvalidValue, "cuTensorMapEncodeTiled");
  }
  char* w = static_cast<char*>(workspace);
  a.err = reinterpret_cast<int*>(w);
  a.cta_err = reinterpret_cast<int*>(w + L.err);
  a.part_o = reinterpret_cast<float*>(w + L.part_o);
  a.part_ml = reinterpret_cast<float*>(w + L.part_ml);
  if (cache->mass) {
    a.lse2 = reinterpret_cast<float*>(w + L.lse2);
    a.scores = reinterpret_cast<float*>(w + L.scores);
    a.score_pitch = L.pitch;
    a.mass4 = cache->page_size % 4 == 0 && reinterpret_cast<uintptr_t>(cache->mass) % 16 == 0;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dtype == SAGE_F16)
    e = head_dim <= 64 ? launch_decode_t<__half, 64>(a, maps, st) : launch_decode_t<__half, 128>(a, maps, st);
  else
    e = head_dim <= 64 ? launch_decode_t<__nv_bfloat16, 64>(a, maps, st) : launch_decode_t<__nv_bfloat16, 128>(a, maps, st);
  return e == cudaSuccess ? SAGE_OK : note_cuda_failure(e, "paged attention");
}

}  // extern "C"
