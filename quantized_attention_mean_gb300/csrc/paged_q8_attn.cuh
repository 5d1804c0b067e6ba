// The decode kernel over an 8-bit paged cache (sage_paged_attn_q8) and its launch.
//
//   t_j = sm_scale s_k(j) q.c_k(j), capped to cap tanh(t_j / cap), less slope |pos_q - j|
//   out = sum_j softmax(t)_j s_v(j) c_v(j),  lse = ln sum_j exp t_j;  c: codes, s: their blocks' scales
//
// DRAM bounds it, at half the bytes of 16-bit rows, so per byte twice as many instructions are spent as by the kernel
// over those. What keeps them few:
// - The products are transposed: keys (then channels) are the 16 rows of m16n8k16, the query heads of a key/value head its
//   8 columns, so that the usual groups of 4 to 8 heads fill an instruction that they would half leave empty as rows.
// - Codes become fp16 in registers, exactly (an E4M3 code by one conversion per pair, an int8 code as 1024 + code + 128
//   by a byte permutation and one subtraction); scales are applied to scores and weights, one per key, never to codes.
// - q becomes fp16 scaled by a power of two, which takes the largest channel of its row to [2^14, 2^15): channels down to
//   2^-38 of it keep the bits they have, so nothing is lost against bf16.
// - V's scale goes into the weight before it is rounded to fp16, w = 2^(t + log2 s_v - F), with F a running frame of
//   t + log2 s_v of its own: weights of blocks with small scales keep their bits, whatever the largest scale is. Results of warps,
//   clusters and ranges are joined by their F, sums by their m.
// - Rows and columns change places between the products by movmatrix; V is read transposed by ldmatrix, two keys by two
//   channels in a register, of which a byte permutation makes the pairs of keys that the product wants.
//
// 32 sequences of 0.1 to 32K tokens, 32 / 8 heads of head_dim 128 (1.11 GB): 184 us, 6.0 TB/s, 89% of a copy; two of 50 to 60K tokens, 32
// heads of 64, biased: 97 us, 4.8 TB/s, of which 18 us are start, join and the CTAs' uneven ends; one of 1000 tokens: 7.4 us.
//
// Split, loads and join as in the kernel over 16-bit rows (decode_line.cuh): ranges of one line of items, or clusters
// of eight CTAs where heads are few and sequences short.
#pragma once
#include "decode_line.cuh"
#include "launch.h"
#include "paged_q8.cuh"

namespace sage {

struct Q8Args {
  DecodeArgs a;
  const float* ks; const float* vs;
  int block, blocks;
  int block_shift;  // log2 of block, or -1
  int unit;      // bytes of one copy where rows do not come by TMA: 16, 8, 4, or 1 (plain loads)
  int bf16;      // type of q and out
  int q4;        // q allows accesses of four channels
  int o_run;     // out allows accesses of dp / 16 channels
  int cluster;   // form: clusters, or the line
  int k_type, v_type;
};

cudaError_t launch_q8_decode_64(const Q8Args& p, const CUtensorMap* maps, cudaStream_t st);
cudaError_t launch_q8_decode_128(const Q8Args& p, const CUtensorMap* maps, cudaStream_t st);

// NH: blocks of eight query heads, the columns of the products. Up to eight heads, and sixteen of head_dim 64, leave registers
// for three CTAs per SM with two stages each, sixteen of 128 take two CTAs with three stages (three: 146 us against 119).
template <int DP, int NH>
struct Q8Cfg {
  static constexpr int kPerSm = NH == 1 || DP == 64 ? 3 : 2;
  static constexpr int kRanges = 152 * kPerSm;                // of the line
  static constexpr int kStages = kPerSm == 3 ? 2 : 3;
  // keys of a step, whose scores are in registers: 64 of sixteen heads would need more of those and twice the code (16
  // sequences of 30K tokens, head_dim 64: 145 us against 132), of eight heads they are faster (104 against 109)
  static constexpr int kStep = DP == 64 && NH == 1 ? 64 : 32;
  static constexpr int kKeys = DP == 128 ? 32 : 64;           // keys per warp and tile (8 KB of K and V)
  static constexpr int kTile = 4 * kKeys;                     // keys per tile
  static constexpr int kTileBytes = kKeys * DP;               // K or V of one warp's tile
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kWarpBytes = kStages * kStageBytes;
  static constexpr int kOffScale = 4 * kWarpBytes;
  static constexpr int kOffMl = kOffScale + 4 * kStages * 2 * kKeys * 4;
  static constexpr int kOffBar = kOffMl + 4 * 16 * 4 * 4;
  static constexpr int kSmem = kOffBar + 4 * kStages * 8;
};

namespace {

template <int N>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void* src, int src_bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(src_bytes) : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ float lg2_approx(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Four codes as two pairs of fp16: bytes (A, B) and (C, D) of x.
template <int TYPE, int A, int B, int C, int D>
__device__ __forceinline__ void widen(uint32_t x, uint32_t& lo, uint32_t& hi) {
  if constexpr (TYPE == SAGE_S8) {
    const uint32_t u = x ^ 0x80808080u;  // code + 128
    const __half2 bias = __half2half2(__ushort_as_half(0x6480));  // 1024 + 128
    const uint32_t a = __byte_perm(u, 0x64646464u, A | 4 << 4 | B << 8 | 4 << 12);
    const uint32_t b = __byte_perm(u, 0x64646464u, C | 4 << 4 | D << 8 | 4 << 12);
    const __half2 ha = __hsub2(*reinterpret_cast<const __half2*>(&a), bias);
    const __half2 hb = __hsub2(*reinterpret_cast<const __half2*>(&b), bias);
    lo = *reinterpret_cast<const uint32_t*>(&ha);
    hi = *reinterpret_cast<const uint32_t*>(&hb);
  } else {
    const uint32_t u = A == 0 && B == 1 ? x : __byte_perm(x, 0, A | B << 4 | C << 8 | D << 12);
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(u));
  }
}
// Whether a stage's boxes have landed.
__device__ __forceinline__ bool ready(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Byte offset of 16-byte unit c of row r of a tile: the swizzle that a TMA box of rows of DP bytes is written with.
template <int DP>
__device__ __forceinline__ int unit_at(int r, int c) {
  return DP == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

// A warp's keys of one item into a stage: K, V and the keys' scales. Tokens that are not there and channels past d become
// zero. page, slot: of keys lane, lane + 32, ...
template <typename C, int DP, int KS, int N>
__device__ __forceinline__ void load_q8_stage(const Q8Args& p, const CUtensorMap* tmK, const CUtensorMap* tmV, int h,
                                              const int (&page)[N], const int (&slot)[N], uint8_t* stage, float* scale,
                                              uint32_t bar) {
  const DecodeArgs& a = p.a;
  const int lane = threadIdx.x & 31;
  const uint32_t base = smem_u32(stage);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const bool in = page[i] >= 0;
    const int blk = p.block_shift >= 0 ? slot[i] >> p.block_shift : slot[i] / p.block;
    const int64_t at = in ? ((int64_t)page[i] * a.c.hkv + h) * p.blocks + blk : 0;
    const uint32_t dst = smem_u32(scale + lane + 32 * i);
    cp_async_small<4>(dst, p.ks + at, in ? 4 : 0);
    cp_async_small<4>(dst + C::kKeys * 4, p.vs + at, in ? 4 : 0);
  }
  if (a.load == kLoadTma) {
    // issued by one elected lane with operands that all lanes agree on: lanes with boxes of their own would take turns
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar), "r"(C::kStageBytes)
        : "memory");
#pragma unroll 1
    for (int row = 0; row < C::kKeys; row += a.box_rows) {
      int pg = __shfl_sync(0xffffffffu, page[0], row & 31), sl = __shfl_sync(0xffffffffu, slot[0], row & 31);
      if (N > 1 && row >= 32) {
        pg = __shfl_sync(0xffffffffu, page[N - 1], row & 31);
        sl = __shfl_sync(0xffffffffu, slot[N - 1], row & 31);
      }
      pg = pg >= 0 ? pg : a.c.num_pages;  // (outside of the tensor: zeros)
      asm volatile(
          "{\n\t.reg .pred e;\n\t"
          "elect.sync _|e, 0xffffffff;\n\t"
          "@e cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%2, {%5, %6, %7, %8}], [%4];\n\t"
          "@e cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%1], [%3, {%5, %6, %7, %8}], [%4];\n\t}" ::"r"(
              base + row * DP),
          "r"(base + C::kTileBytes + row * DP), "l"(reinterpret_cast<uint64_t>(tmK)), "l"(reinterpret_cast<uint64_t>(tmV)), "r"(bar),
          "r"(0), "r"(sl), "r"(h), "r"(pg)
          : "memory");
    }
    return;
  }
  // rows' places, of keys lane, lane + 32, ..., which the lanes that copy a row ask for
  const uint8_t* kb = static_cast<const uint8_t*>(a.c.k) + h * a.c.k_sh;
  const uint8_t* vb = static_cast<const uint8_t*>(a.c.v) + h * a.c.v_sh;
  long long ko[N], vo[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    ko[i] = page[i] >= 0 ? page[i] * a.c.k_sp + slot[i] * a.c.k_st : -1;
    vo[i] = page[i] >= 0 ? page[i] * a.c.v_sp + slot[i] * a.c.v_st : -1;
  }
  auto copy = [&](auto unit) {
    // a lane takes 16 bytes of a row, in copies of U
    constexpr int U = decltype(unit)::value, kUnits = KS == 6 ? 8 : KS, kRowsPer = 32 / kUnits;
    const int c = lane % kUnits, r0 = lane / kUnits, left = a.c.d - c * 16;
#pragma unroll 2
    for (int i = 0; i < C::kKeys / kRowsPer; ++i) {
      const int r = i * kRowsPer + r0;
      long long kr = __shfl_sync(0xffffffffu, ko[0], r & 31), vr = __shfl_sync(0xffffffffu, vo[0], r & 31);
      if (N > 1 && i * kRowsPer >= 32) {
        kr = __shfl_sync(0xffffffffu, ko[N - 1], r & 31);
        vr = __shfl_sync(0xffffffffu, vo[N - 1], r & 31);
      }
      const int n = kr >= 0 ? left : 0;
      const uint32_t dst = base + unit_at<DP>(r, c);
      const uint8_t *ks = n > 0 ? kb + kr + c * 16 : kb, *vs = n > 0 ? vb + vr + c * 16 : vb;
#pragma unroll
      for (int e = 0; e < 16; e += U) {
        const int bytes = n > e ? U : 0;
        const uint8_t *kf = bytes ? ks + e : kb, *vf = bytes ? vs + e : vb;
        if constexpr (U == 16) {
          cp_async16(dst, kf, bytes);
          cp_async16(dst + C::kTileBytes, vf, bytes);
        } else {
          cp_async_small<U>(dst + e, kf, bytes);
          cp_async_small<U>(dst + C::kTileBytes + e, vf, bytes);
        }
      }
    }
  };
  if (p.unit == 16) copy(std::integral_constant<int, 16>{});
  else if (p.unit == 8) copy(std::integral_constant<int, 8>{});
  else if (p.unit == 4) copy(std::integral_constant<int, 4>{});
  else {
    // byte by byte: a row takes several turns of the warp
#pragma unroll 1
    for (int r = 0; r < C::kKeys; ++r) {
      long long kr = __shfl_sync(0xffffffffu, ko[0], r & 31), vr = __shfl_sync(0xffffffffu, vo[0], r & 31);
      if (N > 1 && r >= 32) {
        kr = __shfl_sync(0xffffffffu, ko[N - 1], r & 31);
        vr = __shfl_sync(0xffffffffu, vo[N - 1], r & 31);
      }
#pragma unroll
      for (int c = lane; c < KS * 16; c += 32) {
        const bool in = kr >= 0 && c < a.c.d;
        const int off = unit_at<DP>(r, c / 16) + c % 16;
        stage[off] = in ? kb[kr + c] : 0;
        stage[C::kTileBytes + off] = in ? vb[vr + c] : 0;
      }
    }
  }
}

__device__ __forceinline__ void store_out(const Q8Args& p, int64_t at, float x) {
  if (p.bf16) static_cast<__nv_bfloat16*>(p.a.o)[at] = __float2bfloat16_rn(x);
  else static_cast<__half*>(p.a.o)[at] = __float2half_rn(x);
}

// A run of a row's channels, of which `left` are there, times f.
template <int N>
__device__ __forceinline__ void store_run(const Q8Args& p, int64_t at, int left, const float (&y)[N], float f) {
  if (p.o_run && left >= N) {
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N; i += 2) w[i / 2] = p.bf16 ? pack2<__nv_bfloat16>(y[i] * f, y[i + 1] * f) : pack2<__half>(y[i] * f, y[i + 1] * f);
    void* to = static_cast<uint16_t*>(p.a.o) + at;
    if constexpr (N == 8) *static_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
    else *static_cast<uint2*>(to) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < left) store_out(p, at + i, y[i] * f);
  }
}

// DP: bytes of a row in shared memory; KS: units of 16 channels that the products take.
template <int KT, int VT, int DP, int NH, int KS>
__global__ void __launch_bounds__(kWarps * 32, Q8Cfg<DP, NH>::kPerSm)
    q8_decode_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const __grid_constant__ Q8Args p) {
  using C = Q8Cfg<DP, NH>;
  constexpr int S = C::kStages, M = C::kStep / 16, NP = C::kKeys / 32;
  constexpr float kHead = 7.0f;  // weights are held at up to 2^(7 + 8), so that the smallest keep their bits in fp16
  constexpr float kLeastFrame = -3.4028234e38f;  // of no key: finite, so that differences are numbers
  constexpr float kLeastLog = -110.0f;  // smaller scales do not lower the frame of the weights, which stays finite
  extern __shared__ __align__(1024) uint8_t sm[];
  __shared__ int s_err[kWarps];
  const DecodeArgs& a = p.a;
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // (one value for the warp)
  // an item is a tile of `side` heads that lie side by side: warps of one head share its keys
  const int side = a.side, sub = warp & (side - 1), part = warp / side;
  const int heads = a.c.hkv / side * a.row_blocks;
  uint8_t* const ring = sm + warp * C::kWarpBytes;
  float* const scales = reinterpret_cast<float*>(sm + C::kOffScale) + warp * S * 2 * C::kKeys;
  float4* const ml = reinterpret_cast<float4*>(sm + C::kOffMl);  // [warp][row]: m, l, F
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
  int left = 0;  // (of the line's items, of which this CTA's range has far fewer than 2^31)
  Cursor cu{a.c.batch, 0, 0, 1, 0};
  __shared__ long long s_base;
  __shared__ int s_b;
  if (p.cluster) {
    const int rank = me % kRanks;
    cu.b = blockIdx.y;
    cu.h = me / kRanks;
    cu.len = max(checked_len(a.c, cu.b, a.max_len), 0);
    cu.tiles = tiles_of(cu.len, a.tile_shift);
    cu.tile = cu.tiles * rank / kRanks;
    left = cu.tiles * (rank + 1) / kRanks - cu.tile;
  } else {
    // this CTA's range of the line: the total, then the sequence that its first item lies in
    bool bad = false;
    if (threadIdx.x == 0) { s_b = a.c.batch; s_base = 0; }
    Scan sc = scan_items(a, a.tile_shift, heads, 0, bad);
    long long total = sc.all;
    for (int b0 = blockDim.x; b0 < a.c.batch; b0 += blockDim.x) total += scan_items(a, a.tile_shift, heads, b0, bad).all;
    const int ctas = total > 0 ? ctas_of<C::kRanges>(total) : 0;
    long long i0 = 0;
    if (me < ctas) {
      i0 = first_item(total, ctas, me);
      left = (int)(first_item(total, ctas, me + 1) - i0);
      long long base = 0;
      for (int b0 = 0;;) {
        const long long lo = base + sc.before;
        if (sc.n > 0 && i0 >= lo && i0 < lo + sc.n) { s_b = b0 + threadIdx.x; s_base = lo; }
        base += sc.all;
        b0 += blockDim.x;
        if (base > i0 || b0 >= a.c.batch) break;
        sc = scan_items(a, a.tile_shift, heads, b0, bad);
      }
    }
    __syncthreads();
    err = bad ? kDevSeqlens : 0;
    if (left > 0) {
      cu.b = s_b;
      cu.len = checked_len(a.c, cu.b, a.max_len);
      cu.tiles = tiles_of(cu.len, a.tile_shift);
      const long long in = i0 - s_base;
      cu.h = (int)(in / cu.tiles);
      cu.tile = (int)(in - (long long)cu.h * cu.tiles);
    }
  }
  pdl_trigger();
  if (p.cluster && a.err && me == 0 && blockIdx.y == 0) {
    // the status word has one writer (but for a wait that runs out, two seconds from now): the first
    // CTA looks at the lengths and pages of all sequences
    int e = 0;
    for (int b = 0; b < a.c.batch; ++b) {
      const int len = checked_len(a.c, b, a.max_len);
      if (len < 0) e = max(e, (int)kDevSeqlens);
      for (int64_t i = threadIdx.x; i < ((int64_t)len + a.c.page_size - 1) / a.c.page_size; i += kWarps * 32) {
        const int pg = __ldg(&a.c.table[b * a.c.table_stride + i]);
        if (pg < 0 || pg >= a.c.num_pages) e = max(e, kDevPage);
      }
    }
    e = __reduce_max_sync(0xffffffffu, e);
    if (lane == 0) s_err[warp] = e;
    __syncthreads();
    if (threadIdx.x == 0) *a.err = max(max(s_err[0], s_err[1]), max(s_err[2], s_err[3]));
  }
  // ---- fill the ring: S - 1 stages in flight, the pages of the stage after them already read
  Cursor ld = cu;
  int to_load = left;
  int page[NP], slot[NP];
  auto next_page = [&]() {
    const int* const row = a.c.table + ld.b * a.c.table_stride;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int key = (ld.tile << a.tile_shift) + part * C::kKeys + i * 32 + lane, at = page_index(a, key);
      const bool live = to_load > 0 && key < ld.len;
      slot[i] = key - at * a.c.page_size;
      page[i] = live ? __ldg(row + at) : -1;
      const bool bad = live && (unsigned)page[i] >= (unsigned)a.c.num_pages;
      page[i] = bad ? -1 : page[i];
      err = bad ? kDevPage : err;
    }
  };
  bool dead = false;  // a wait has run out: nothing more is loaded
  auto load_next = [&](int st) {
    if (to_load > 0 && !dead) {
      const int h = a.row_blocks == 1 ? ld.h : ld.h / a.row_blocks;
      load_q8_stage<C, DP, KS>(p, &tmK, &tmV, h * side + sub, page, slot, ring + st * C::kStageBytes,
                        scales + st * 2 * C::kKeys, bars + st * 8);
      next_item(a, a.tile_shift, heads, ld);
      --to_load;
      next_page();
    }
    cp_async_commit();
  };
  __syncwarp();
  next_page();
#pragma unroll 1
  for (int st = 0; st < S - 1; ++st) load_next(st);

  // columns of this thread: heads 8 x + 2 (lane & 3) + e; rows of a fragment: lane >> 2 and + 8
  const int r0 = lane >> 2, j = lane & 3;
  float o[KS][NH][4], m[NH][2], F[NH][2], l[NH][2], qs[NH][2], sl[NH][2];
  uint32_t qf[KS][NH][2];
  int qpos = 0, rows = 0, row0 = 0, tile0 = 0, pieces = 0;
  bool fresh = true;
  float gap = 0.f;
  if (p.cluster) {
    const int rb = cu.h % a.row_blocks;
    row0 = cu.h / a.row_blocks * a.group + rb * kRows;
    rows = min(kRows, a.group - rb * kRows);
  }
  const float factor = a.cap > 0.f ? a.sm_scale / a.cap : a.sm_scale * kLog2eF, cap_out = a.cap * kLog2eF;
  int stage = 0;
  uint32_t parity = 0;

#pragma unroll 1
  for (; left > 0; --left) {
    if (fresh) {
      // a new (sequence, head): its query rows as the B operand, its statistics
      fresh = false;
      tile0 = cu.tile;
      const int h = cu.h / a.row_blocks, rb = cu.h - h * a.row_blocks;
      row0 = (h * side + sub) * a.group + rb * kRows;
      rows = min(kRows, a.group - rb * kRows);
#pragma unroll
      for (int x = 0; x < NH; ++x) {
        const int r = x * 8 + r0;
        const int64_t at = cu.b * a.q_sb + (int64_t)(row0 + r) * a.q_sh;
        float most = 0.f;
        uint2 raw[KS];
#pragma unroll
        for (int u = 0; u < KS; ++u) {
          // channels 16 u + 4 j .. + 3: the places 2 j, 2 j + 1, 2 j + 8 and 2 j + 9 of the product's sum
          const int c = u * 16 + j * 4;
          raw[u] = make_uint2(0, 0);
          if (r < rows && c < a.c.d) {
            const uint16_t* src = static_cast<const uint16_t*>(a.q) + at + c;
            if (p.q4) {
              raw[u] = *reinterpret_cast<const uint2*>(src);
            } else {
              uint16_t t[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) t[e] = c + e < a.c.d ? src[e] : 0;
              raw[u] = make_uint2(t[0] | (uint32_t)t[1] << 16, t[2] | (uint32_t)t[3] << 16);
            }
          }
        }
        auto value = [&](uint32_t w, int hi) {
          const uint16_t b = (uint16_t)(hi ? w >> 16 : w);
          return p.bf16 ? __uint_as_float((uint32_t)b << 16) : __half2float(__ushort_as_half(b));
        };
#pragma unroll
        for (int u = 0; u < KS; ++u)
          most = fmaxf(fmaxf(most, fmaxf(fabsf(value(raw[u].x, 0)), fabsf(value(raw[u].x, 1)))),
                       fmaxf(fabsf(value(raw[u].y, 0)), fabsf(value(raw[u].y, 1))));
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
        // the row times 2^(14 - e), e the exponent of its largest channel
        const int e = max(16, min(254, (int)(__float_as_uint(most) >> 23)));
        const float up = __uint_as_float((uint32_t)(268 - e) << 23), down = __uint_as_float((uint32_t)(e - 14) << 23);
#pragma unroll
        for (int u = 0; u < KS; ++u) {
          qf[u][x][0] = pack2<__half>(value(raw[u].x, 0) * up, value(raw[u].x, 1) * up);
          qf[u][x][1] = pack2<__half>(value(raw[u].y, 0) * up, value(raw[u].y, 1) * up);
        }
#pragma unroll
        for (int e2 = 0; e2 < 2; ++e2) {
          qs[x][e2] = __shfl_sync(0xffffffffu, down, (2 * j + e2) * 4) * factor;
          const int rr = x * 8 + 2 * j + e2;
          sl[x][e2] = a.slopes && rr < rows ? __ldg(&a.slopes[row0 + rr]) * kLog2eF : 0.f;
          m[x][e2] = F[x][e2] = kLeastFrame;
          l[x][e2] = 0.f;
        }
#pragma unroll
        for (int u = 0; u < KS; ++u) o[u][x][0] = o[u][x][1] = o[u][x][2] = o[u][x][3] = 0.f;
      }
      qpos = a.q_pos ? __ldg(&a.q_pos[cu.b]) : cu.len - 1;
    }
    // the stage after the ones in flight goes where the previous item was
    __syncwarp();
    load_next(stage == 0 ? S - 1 : stage - 1);
    const int key0 = (cu.tile << a.tile_shift) + part * C::kKeys;
    uint8_t* const here = ring + stage * C::kStageBytes;
    const float* const sc = scales + stage * 2 * C::kKeys;
    if (a.load == kLoadTma) {
      if (!dead && !__all_sync(0xffffffffu, ready(bars + stage * 8, parity)) &&
          !__all_sync(0xffffffffu, wait_stage(bars + stage * 8, parity))) {
        dead = true;
        err = kDevTimeout;
        // what is in flight lands (or runs out of time) before the shared memory goes away
        for (int k = 0; k < left - to_load; ++k) {
          const int st = stage + k;
          wait_stage(bars + (st % S) * 8, parity ^ (st >= S ? 1u : 0u));
        }
      }
      if (VT == SAGE_E4M3 && !dead && key0 < cu.len && key0 + C::kKeys > cu.len) {
        // slots behind the last token may hold anything, a NaN too: as V rows they become zero (their scores are masked)
        for (int i = lane; i < (key0 + C::kKeys - cu.len) * (DP / 16); i += 32)
          *reinterpret_cast<uint4*>(here + C::kTileBytes + (cu.len - key0 + i / (DP / 16)) * DP + i % (DP / 16) * 16) =
              make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
      }
    }
    cp_async_wait<S - 1>();
    __syncwarp();
#pragma unroll 1
    for (int k0 = 0; k0 < C::kKeys && key0 + k0 < cu.len; k0 += C::kStep) {
      // (keys 0-15 at unit u = 0, then at unit 1: other units by exclusive or, which the swizzle is)
      const uint32_t kb = smem_u32(here) + k0 * DP + unit_at<DP>(lane & 15, lane >> 4);
      // ---- S^T = K Q^T: 16 keys x 8 heads each
      float s[M][NH][4];
#pragma unroll
      for (int g = 0; g < M; ++g)
#pragma unroll
        for (int x = 0; x < NH; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[g][x][e] = 0.f;
      {
#pragma unroll
        for (int u = 0; u < KS; u += 2)
#pragma unroll
          for (int g = 0; g < M; ++g) {
            uint32_t b[4], f[4];
            ldsm4((kb ^ (u << 4)) + g * 16 * DP, b);
            widen<KT, 0, 1, 2, 3>(b[0], f[0], f[2]);
            widen<KT, 0, 1, 2, 3>(b[1], f[1], f[3]);
#pragma unroll
            for (int x = 0; x < NH; ++x) mma16816<__half>(s[g][x], f, qf[u][x][0], qf[u][x][1]);
            widen<KT, 0, 1, 2, 3>(b[2], f[0], f[2]);
            widen<KT, 0, 1, 2, 3>(b[3], f[1], f[3]);
#pragma unroll
            for (int x = 0; x < NH; ++x) mma16816<__half>(s[g][x], f, qf[u + 1][x][0], qf[u + 1][x][1]);
          }
      }
      // ---- scores in base 2; s[g][x][2 b + e]: key 16 g + 8 b + r0, head 8 x + 2 j + e
      float sv[M][2];  // V's scales
      float most = 0.f;
#pragma unroll
      for (int g = 0; g < M; ++g)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const float ks = sc[k0 + g * 16 + b * 8 + r0];
          sv[g][b] = sc[C::kKeys + k0 + g * 16 + b * 8 + r0];
          most = fmaxf(most, sv[g][b]);
#pragma unroll
          for (int x = 0; x < NH; ++x)
#pragma unroll
            for (int e = 0; e < 2; ++e) s[g][x][2 * b + e] *= qs[x][e] * ks;
        }
      if (a.cap > 0.f) {
#pragma unroll
        for (int g = 0; g < M; ++g)
#pragma unroll
          for (int x = 0; x < NH; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[g][x][e] = tanhf(s[g][x][e]) * cap_out;
      }
      if (a.slopes) {
        const float d0 = (float)((long long)qpos - (key0 + k0 + r0));  // exact below 2^24
#pragma unroll
        for (int g = 0; g < M; ++g)
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const float dist = fabsf(d0 - (float)(g * 16 + b * 8));
#pragma unroll
            for (int x = 0; x < NH; ++x)
#pragma unroll
              for (int e = 0; e < 2; ++e) s[g][x][2 * b + e] = fmaf(-sl[x][e], dist, s[g][x][2 * b + e]);
          }
      }
      if (key0 + k0 + C::kStep > cu.len) {
#pragma unroll
        for (int g = 0; g < M; ++g)
#pragma unroll
          for (int x = 0; x < NH; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (key0 + k0 + g * 16 + (e >> 1) * 8 + r0 >= cu.len) s[g][x][e] = -INFINITY;
      }
      // a lane's largest score t, and a bound of its t + log2 s_v: the largest score with the largest scale
      const float lv = fmaxf(lg2_approx(most), kLeastLog);
      float tm[NH][2], um[NH][2];
#pragma unroll
      for (int x = 0; x < NH; ++x)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          tm[x][e] = fmaxf(s[0][x][e], s[0][x][2 + e]);
#pragma unroll
          for (int g = 1; g < M; ++g) tm[x][e] = max3(tm[x][e], s[g][x][e], s[g][x][2 + e]);
          um[x][e] = tm[x][e] + lv;
        }
      // ---- frames of the sum (m) and of the weights (F, kHead below the largest); `gap`: the largest m - F. The eight lanes of a
      // head agree. Frames are kept unless a maximum grew by more than 8, so sums and O are rescaled rarely
      const float top = fminf(100.0f - lv, 126.0f);
      bool grows = gap > top, far = false;
#pragma unroll
      for (int x = 0; x < NH; ++x)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          grows |= tm[x][e] > m[x][e] + 8.0f || um[x][e] > F[x][e] + (8.0f + kHead);
      if (__any_sync(0xffffffffu, grows)) {
        // (the bound may say so in vain where a lane's scales differ; a frame above the largest weight would cost the small ones
        // their bits)
        float least = sv[0][0];
#pragma unroll
        for (int g = 0; g < M; ++g) least = fminf(least, fminf(sv[g][0], sv[g][1]));
        if (__any_sync(0xffffffffu, least < most)) {
#pragma unroll
          for (int x = 0; x < NH; ++x) um[x][0] = um[x][1] = -INFINITY;
#pragma unroll
          for (int g = 0; g < M; ++g)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              const float l2 = fmaxf(lg2_approx(sv[g][b]), kLeastLog);
#pragma unroll
              for (int x = 0; x < NH; ++x) {
                um[x][0] = fmaxf(um[x][0], s[g][x][2 * b] + l2);
                um[x][1] = fmaxf(um[x][1], s[g][x][2 * b + 1] + l2);
              }
            }
        }
#pragma unroll
        for (int x = 0; x < NH; ++x)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float t = tm[x][e], v = um[x][e];
#pragma unroll
            for (int w = 4; w < 32; w <<= 1) {
              t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, w));
              v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, w));
            }
            v -= kHead;
            if (t > m[x][e]) {
              l[x][e] *= ex2_approx(m[x][e] - t);
              m[x][e] = t;
            }
            if (v > F[x][e]) {
              const float f = ex2_approx(F[x][e] - v);
              F[x][e] = v;
#pragma unroll
              for (int u = 0; u < KS; ++u) {
                o[u][x][e] *= f;
                o[u][x][2 + e] *= f;
              }
            }
          }
        gap = m[0][0] - F[0][0];
#pragma unroll
        for (int x = 0; x < NH; ++x)
#pragma unroll
          for (int e = 0; e < 2; ++e) gap = fmaxf(gap, m[x][e] - F[x][e]);
        far = __any_sync(0xffffffffu, gap > top);
        if (far) {
          // the sums; then t + log2 s_v - F - 100 in the place of t - m, which adds nothing to them, and 2^100 in that of the scale
#pragma unroll
          for (int g = 0; g < M; ++g)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              const float l2 = lg2_approx(sv[g][b]) - 100.0f;
              sv[g][b] = 0x1p100f;
#pragma unroll
              for (int x = 0; x < NH; ++x)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  float& t = s[g][x][2 * b + e];
                  l[x][e] += ex2_approx(t - m[x][e]);
                  t = t + (m[x][e] - F[x][e]) + l2;
                }
            }
        }
      }
      // ---- weights p = 2^(t - m): their sum in 32 bits; as p s_v 2^(m - F) rounded once, keys and heads exchanged, the B
      // operand. That product is good while 2^(m - F) times the largest scale stays below 2^100: p too small for fp32 are then
      // too small for fp16 as weights. Past that (`far`: scales that outweigh scores 85 and more below the top one) weights are
      // formed as 2^(t + log2 s_v - F), which the logarithm puts off by 2^-15 at most
      uint32_t pf[M][NH][2];
#pragma unroll
      for (int x = 0; x < NH; ++x) {
        const float m0 = m[x][0], m1 = m[x][1];
        const float g0 = ex2_approx(m0 - (far ? m0 : F[x][0])), g1 = ex2_approx(m1 - (far ? m1 : F[x][1]));
#pragma unroll
        for (int g = 0; g < M; ++g)
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const float p0 = ex2_approx(s[g][x][2 * b] - m0), p1 = ex2_approx(s[g][x][2 * b + 1] - m1);
            l[x][0] += p0;
            l[x][1] += p1;
            pf[g][x][b] = transpose8x8(pack2<__half>(p0 * (sv[g][b] * g0), p1 * (sv[g][b] * g1)));
          }
      }
      // ---- O^T += V^T P^T: 16 channels x 8 heads each, 16 keys at a time. Row r0 of a fragment is channel 2 r0 of its
      // unit, row r0 + 8 channel 2 r0 + 1: the two channels of a register that the transposed read gives
      {
#pragma unroll
        for (int g = 0; g < M; ++g)
#pragma unroll
          for (int u = 0; u < KS; u += 2) {
            uint32_t b[4], f[4];
            ldsm4t((kb ^ (u << 4)) + C::kTileBytes + g * 16 * DP, b);
            widen<VT, 0, 2, 1, 3>(b[0], f[0], f[1]);
            widen<VT, 0, 2, 1, 3>(b[1], f[2], f[3]);
#pragma unroll
            for (int x = 0; x < NH; ++x) mma16816<__half>(o[u][x], f, pf[g][x][0], pf[g][x][1]);
            widen<VT, 0, 2, 1, 3>(b[2], f[0], f[1]);
            widen<VT, 0, 2, 1, 3>(b[3], f[2], f[3]);
#pragma unroll
            for (int x = 0; x < NH; ++x) mma16816<__half>(o[u + 1][x], f, pf[g][x][0], pf[g][x][1]);
          }
      }
    }
    if (stage + 1 == S) {
      stage = 0;
      parity ^= 1;
    } else {
      ++stage;
    }
    if (!p.cluster && (cu.tile + 1 == cu.tiles || left == 1)) {
      // ---- merge the warps: sums of a head over its eight lanes; each warp's accumulator goes where its last tile was,
      // then every thread sums a run of channels of one head's row over the warps, in their order
      constexpr int P = DP + 8, kRun = DP / 16;  // (the pitch takes the rows of a store to other banks)
      const int past = (stage == 0 ? S - 1 : stage - 1) * C::kStageBytes;
#pragma unroll
      for (int x = 0; x < NH; ++x)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int w = 4; w < 32; w <<= 1) l[x][e] += __shfl_xor_sync(0xffffffffu, l[x][e], w);
          if (r0 == 0) ml[warp * kRows + x * 8 + 2 * j + e] = make_float4(m[x][e], l[x][e], F[x][e], 0.f);
        }
      // the whole (sequence, head) in this range: the result; a part of it: to the workspace
      const bool whole = tile0 == 0 && cu.tile + 1 == cu.tiles;
      const int hg = a.row_blocks == 1 ? cu.h : cu.h / a.row_blocks, rb = cu.h - hg * a.row_blocks;
      float* const mine = reinterpret_cast<float*>(ring + past);
      const int at_row = threadIdx.x >> 4, c = (threadIdx.x & 15) * kRun;
#pragma unroll
      for (int x = 0; x < NH; ++x) {
#pragma unroll
        for (int u = 0; u < KS; ++u)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            *reinterpret_cast<float2*>(mine + (2 * j + e) * P + u * 16 + 2 * r0) = make_float2(o[u][x][e], o[u][x][2 + e]);
        __syncthreads();
        const int r = x * 8 + at_row;
        if (r < rows && c < KS * 16) {
#pragma unroll 1
          for (int t = 0; t < side; ++t) {
            const float4* st = ml + t * kRows + r;
            float mm = -INFINITY, ff = -INFINITY, ll = 0.f, y[kRun];
            for (int w = 0; w < kWarps; w += side) {
              mm = fmaxf(mm, st[w * kRows].x);
              ff = fmaxf(ff, st[w * kRows].z);
            }
            const float mu = mm == -INFINITY ? 0.f : mm, fu = ff == -INFINITY ? 0.f : ff;
#pragma unroll
            for (int i = 0; i < kRun; ++i) y[i] = 0.f;
            for (int w = 0; w < kWarps; w += side) {
              ll += st[w * kRows].y * ex2_approx(st[w * kRows].x - mu);
              const float f = ex2_approx(st[w * kRows].z - fu);
              const float* from = reinterpret_cast<const float*>(sm + (t + w) * C::kWarpBytes + past) + at_row * P + c;
#pragma unroll
              for (int i = 0; i < kRun; ++i) y[i] = fmaf(f, from[i], y[i]);
            }
            const float f = !whole ? 1.0f : ll != 0.f ? ex2_approx(ff - mu) / ll : 0.f;
            const int row = (hg * side + t) * a.group + rb * kRows + r;
            if (whole) {
              store_run<kRun>(p, cu.b * a.o_sb + (int64_t)row * a.o_sh + c, a.c.d - c, y, f);
              if (c == 0 && a.lse) a.lse[(int64_t)cu.b * a.hq + row] = ll != 0.f ? (mm + log2f(ll)) * kLn2F : -INFINITY;
            } else {
              const int64_t at = (((int64_t)me * 2 + (pieces > 0)) * side + t) * a.part_rows + r;
#pragma unroll
              for (int i = 0; i < kRun; i += 4)
                *reinterpret_cast<float4*>(a.part_o + at * DP + c + i) = make_float4(y[i] * f, y[i + 1] * f, y[i + 2] * f, y[i + 3] * f);
              if (c == 0) *reinterpret_cast<float4*>(a.part_ml + at * 4) = make_float4(mm, ll, ff, 0.f);
            }
          }
        }
        fence_proxy_async_smem();  // (the next tile lands where the accumulators were)
        __syncthreads();
      }
      ++pieces;
      fresh = true;
    }
    next_item(a, a.tile_shift, heads, cu);
  }
  if (p.cluster) {
    // every warp's accumulator into its own ring, its statistics beside; then each thread of the cluster sums one group of
    // four channels of a row over all warps of all ranks, in their order
    constexpr int kParts = kRanks * kWarps, kLanes = DP / 4;  // kLanes: of a row
    const int rank = me % kRanks;
    cp_async_wait<0>();
    __syncwarp();
    float* const mine = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int x = 0; x < NH; ++x)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = x * 8 + 2 * j + e;
        if (!fresh) {
          if (r < rows) {
#pragma unroll
            for (int u = 0; u < KS; ++u)
              *reinterpret_cast<float2*>(mine + r * DP + u * 16 + 2 * r0) = make_float2(o[u][x][e], o[u][x][2 + e]);
          }
#pragma unroll
          for (int w = 4; w < 32; w <<= 1) l[x][e] += __shfl_xor_sync(0xffffffffu, l[x][e], w);
        }
        if (r0 == 0)
          ml[warp * kRows + r] = fresh ? make_float4(-INFINITY, 0.f, -INFINITY, 0.f) : make_float4(m[x][e], l[x][e], F[x][e], 0.f);
      }
    if (dead && a.err) record_error(a.err, kDevTimeout);
    cluster_sync();
    const int cell = rank * kWarps * 32 + threadIdx.x, r = cell / kLanes, c = (cell - r * kLanes) * 4;
    if (__any_sync(0xffffffffu, r < rows)) {
      // the lanes of a row look up the warps' frames side by side
      const uint32_t ml_at = smem_u32(ml + min(r, kRows - 1)), o_at = smem_u32(sm) + (r * DP + c) * 4;
      float4 st[kParts / kLanes];
      float mm = -INFINITY, ff = -INFINITY, ll = 0.f;
#pragma unroll
      for (int i = 0; i < kParts / kLanes; ++i) {
        const int q = i * kLanes + lane % kLanes;
        st[i] = ld_rank4(of_rank(ml_at + (q % kWarps) * kRows * 16, q / kWarps));
        mm = fmaxf(mm, st[i].x);
        ff = fmaxf(ff, st[i].z);
      }
#pragma unroll
      for (int w = kLanes / 2; w > 0; w >>= 1) {
        mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, w));
        ff = fmaxf(ff, __shfl_xor_sync(0xffffffffu, ff, w));
      }
      const float mu = mm == -INFINITY ? 0.f : mm, fu = ff == -INFINITY ? 0.f : ff;
      float in[kParts / kLanes];  // weight of a warp's accumulator
#pragma unroll
      for (int i = 0; i < kParts / kLanes; ++i) {
        ll = fmaf(st[i].y, ex2_approx(st[i].x - mu), ll);
        in[i] = ex2_approx(st[i].z - fu);
      }
#pragma unroll
      for (int w = kLanes / 2; w > 0; w >>= 1) ll += __shfl_xor_sync(0xffffffffu, ll, w);
      const bool on = r < rows && c < KS * 16;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int q = 0; q < kParts; ++q) {
        const float w = __shfl_sync(0xffffffffu, in[q / kLanes], q % kLanes, kLanes);
        if (on && w != 0.f) {  // (a warp without keys wrote no accumulator)
          const float4 y = ld_rank4(of_rank(o_at + (q % kWarps) * C::kWarpBytes, q / kWarps));
          acc.x = fmaf(w, y.x, acc.x); acc.y = fmaf(w, y.y, acc.y);
          acc.z = fmaf(w, y.z, acc.z); acc.w = fmaf(w, y.w, acc.w);
        }
      }
      if (on) {
        const float f = ll != 0.f ? ex2_approx(ff - mu) / ll : 0.f;
        const float y[4] = {acc.x * f, acc.y * f, acc.z * f, acc.w * f};
        const int64_t to = (int64_t)blockIdx.y * a.o_sb + (int64_t)(row0 + r) * a.o_sh + c;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (c + e < a.c.d) store_out(p, to + e, y[e]);
        if (c == 0 && a.lse) a.lse[(int64_t)blockIdx.y * a.hq + row0 + r] = ll != 0.f ? (mm + log2f(ll)) * kLn2F : -INFINITY;
      }
    }
    cluster_sync();  // no CTA's shared memory goes away while it is read
    return;
  }
  cp_async_wait<0>();
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

template <int KT, int VT, int DP, int NH, int KS>
cudaError_t launch_q8_t(const Q8Args& p, const CUtensorMap* maps, cudaStream_t st) {
  using C = Q8Cfg<DP, NH>;
  const DecodeArgs& a = p.a;
  static std::atomic<int> limits[64];
  cudaError_t e = raise_smem_limit(q8_decode_kernel<KT, VT, DP, NH, KS>, C::kSmem, limits);
  if (e != cudaSuccess) return e;
  const int heads = a.c.hkv * a.row_blocks;
  if (!p.cluster) {
    e = launch_pdl(q8_decode_kernel<KT, VT, DP, NH, KS>, dim3(C::kRanges), dim3(kWarps * 32), C::kSmem, st, maps[0], maps[1], p);
    if (e != cudaSuccess) return e;
    const dim3 grid(heads * a.slices, a.c.batch);
    return p.bf16 ? launch_pdl(join_kernel<__nv_bfloat16, DP, C::kRanges, true>, grid, dim3(kJoinThreads), 0, st, a)
                  : launch_pdl(join_kernel<__half, DP, C::kRanges, true>, grid, dim3(kJoinThreads), 0, st, a);
  }
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
  return cudaLaunchKernelEx(&cfg, q8_decode_kernel<KT, VT, DP, NH, KS>, maps[0], maps[1], p);
}

template <int DP>
cudaError_t launch_q8(const Q8Args& p, const CUtensorMap* maps, cudaStream_t st) {
  // head_dims up to 96 and 32 leave out the products of the channels that rows are filled up with (32 x 8000 tokens of
  // head_dim 96: 74 us against 81, of 32: 86 against 99)
  constexpr int kFew = DP == 128 ? 6 : 2;
  const bool wide = p.a.group > 8;
  auto go = [&](auto kt, auto vt) {
    constexpr int K = decltype(kt)::value, V = decltype(vt)::value;
    if (p.a.c.d <= kFew * 16) return wide ? launch_q8_t<K, V, DP, 2, kFew>(p, maps, st) : launch_q8_t<K, V, DP, 1, kFew>(p, maps, st);
    return wide ? launch_q8_t<K, V, DP, 2, DP / 16>(p, maps, st) : launch_q8_t<K, V, DP, 1, DP / 16>(p, maps, st);
  };
  using S8 = std::integral_constant<int, SAGE_S8>;
  using E4 = std::integral_constant<int, SAGE_E4M3>;
  if (p.k_type == SAGE_S8) return p.v_type == SAGE_S8 ? go(S8{}, S8{}) : go(S8{}, E4{});
  return p.v_type == SAGE_S8 ? go(E4{}, S8{}) : go(E4{}, E4{});
}

}  // namespace
}  // namespace sage
