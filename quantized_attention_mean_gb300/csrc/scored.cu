// Attention with modified scores on 16-bit operands (sage_scored_attn): tanh cap, distance bias,
// causal, prefix and document masks.
//
//   s = sm_scale q.k; s = cap tanh(s / cap); s -= slope |i + q_offset - j|; softmax over visible j; times v
//
// One CTA owns two 128-row query tiles (A, B) of one (sequence, head), at head_dim 64 one, and walks the 128-key tiles
// that any of its rows may see. Softmax warps first, then four control warps:
//   softmax   four warps per query tile, one thread per row: S from tensor memory, score modification, mask,
//             running maximum and sum, P to tensor memory
//   control 0 TMA: Q once, then K and V tiles through rings of stages, straight from the caller's tensors
//   control 1 issues the MMAs: S = Q K^T (both operands in shared memory) and O += P V with P in tensor memory and
//             V in its own row order (an MN-major operand), so nothing is transposed
//   control 3 zeroes the V rows that no row of the CTA may see (padding, what lies behind the last key seen) before
//             their tile is multiplied
// head_dim 128: 512 columns hold one S buffer per query tile beside O, and P overlays it. The tiles run half a step
// apart, so that one tile's products run while the other's softmax does; P V may start on the first half of
// P. (With an issuer per tile the two fell into step: 1072 TFLOP/s at 4 x 38 heads of 4096^2, 1250 with one.) One
// query tile alone uses both S buffers in turn.
// head_dim 64: P has columns of its own, and the next scores are computed as soon as the softmax holds the last ones in
// registers. 256 columns, 97 KB and 256 threads let two CTAs share an SM, one's start and end under the other's
// steps (one CTA of two tiles: 628 against 587 us at 4 x 38 heads of 4096^2, 271 against 255 at 8192 causal).
// O is rescaled only when a row's maximum has grown by more than 2^8 since the last rescale: P then stays below 2^8
// (fp16: 2^15, see kHead) and the sum is exact in the same frame, so no precision is lost.
//
// Bound by the softmax warps: per score one exponential (4 cycles a warp and sub-partition), half an instruction each to
// scale, sum and round, and the passes through tensor memory around them; products take 63% of the
// cycles at head_dim 128. Rates (bf16, of 1884 TFLOP/s measured for a library product): 4 x 38 heads of 4096^2, head_dim 128:
// 1490-1500 TFLOP/s, capped 1115-1135, biased 1395; head_dim 64: 1090, capped 645, biased 940. 32 heads of 8 at 8192,
// causal, 128: 368-378 us, capped 505, biased 405, both 566.
// Two costs depend on the values. A product above 0.7 of the cap sends its warp's tile through the loop for masked
// tiles, with the quotient: scores far beyond the cap take 951 us there (head_dim 64: 840 for 450). And fp16 with a cap and a
// slope above 0.32 takes the loop for every tile (see `gentle`): 866 for 566.
#include <cmath>

#include "../../include/sageattn.h"
#include "launch.h"
#include "problem.cuh"
#include "sm103_ptx.cuh"

namespace sage {
namespace {

constexpr float kL2e = 1.4426950408889634f, kL2 = 0.6931471805599453f;
constexpr float kNegInf = -INFINITY;
constexpr int kMaxSplits = 32;

struct DocTile {
  int lo, hi;  // smallest and largest non-negative id; lo > hi: none
  int mixed;   // more than one id, or padding
  int pad;     // some padding
};

// cap tanh(s / cap) for |s| <= 0.7 cap, base 2, as s times a polynomial of s^2: the minimax one of degree 4 of
// tanh(x) / x on [0, 0.7] (found by exchange; tanh is off by at most 2.5e-7 in fp32) with the scales folded in.
// It leaves one exponential per score on the special-function unit, which the quotient's three
// overload. `most`: the largest product |q.k| it is used for (-1: never).
struct CapPoly {
  float c[5], most;
};

struct ScoredArgs {
  int batch, hq, hkv, nq, nk, d, dtype, causal, splits, k_tiles, q_offset, vec;
  // at most 128 queries: a CTA may take several heads of one key/value head, `per_tile` in each query tile, 2^row_bits
  // rows apart; ctas_kv: CTAs per key/value head
  int heads, per_tile, row_bits, ctas_kv;
  float c2;           // sm_scale log2(e)
  float cap2, cap_k;  // cap log2(e); 2 sm_scale log2(e) / cap
  CapPoly poly;
  void* o; int64_t o_sb, o_sh, o_sn;
  float* lse;
  const float* slopes;
  const int* prefix;
  const int* doc_q;
  const int* doc_k;
  // workspace
  int* err;            // status word, or null (no workspace)
  DocTile* doc_tiles;  // [batch][k_tiles]
  float* part_o;       // [splits][batch * hq * nq][dp]
  float* part_ml;      // [splits][batch * hq * nq][2]
};

template <int DP>
struct Cfg {
  static constexpr int kTiles = DP == 128 ? 2 : 1;  // query tiles of a CTA
  static constexpr int kRows = 128 * kTiles, kThreads = kRows + 128, kPerSm = 3 - kTiles;
  static constexpr int kCtl = 4 * kTiles;  // the first of the four control warps
  // the launch's registers, 2 x 128 x 224 + 128 x 56 = 384 x 168 or 128 x 200 + 128 x 56 = 256 x 128
  static constexpr uint32_t kRegsSoft = kTiles == 2 ? 224 : 200, kRegsCtl = 56;
  static constexpr int kChunks = DP / 64;
  static constexpr int kQBytes = 128 * DP * 2, kKBytes = 128 * DP * 2, kVBytes = 128 * DP * 2;
  static constexpr int kKStages = 3, kVStages = 2;
  // tensor memory: S of tile x at 128 x; P over S (head_dim 128) or beside it; then O
  static constexpr bool kOver = DP == 128;
  static constexpr uint32_t kTmemP = kOver ? 0 : 128, kTmemO = kOver ? 256 : 192, kTmemCols = kOver ? 512 : 256;
  static constexpr int kOffK = kTiles * kQBytes, kOffV = kOffK + kKStages * kKBytes;
  static constexpr int kOffBar = kOffV + kVStages * kVBytes;
  static constexpr int kNumBars = 1 + 2 * kKStages + 3 * kVStages + 12;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kSmem = kOffMisc + 128 + 1024;
  static_assert(kTmemO + kTiles * DP <= kTmemCols && kPerSm * (kSmem + 1024) <= 233472, "tensor and shared memory");
};

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcpf(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if constexpr (BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

template <typename F>
__device__ __forceinline__ void each2(float (&t)[16], F f) {
#pragma unroll
  for (int u = 0; u < 16; u += 2) f(t[u], t[u + 1]);
}
// Sixteen products s to cap tanh(s / cap) + (off - cap) in base 2, as off - 2 cap / (1 + e^(2 s / cap)): k = 2 log2(e)
// / cap, m2 = -2 cap.
__device__ __forceinline__ void cap_quotient(float (&t)[16], float k, float m2, float off) {
  each2(t, [&](float& p, float& q) { mul2(p, q, p, q, k, k); });
#pragma unroll
  for (int u = 0; u < 16; ++u) t[u] = ex2f(t[u]);
  each2(t, [&](float& p, float& q) { add2(p, q, p, q, 1.0f, 1.0f); });
#pragma unroll
  for (int u = 0; u < 16; ++u) t[u] = rcpf(t[u]);
  each2(t, [&](float& p, float& q) { fma2(p, q, p, q, m2, m2, off, off); });
}
// Sixteen products to cap tanh(s / cap) by the polynomial.
__device__ __forceinline__ void cap_polynomial(float (&t)[16], const CapPoly& p) {
  float z[16], y[16];
#pragma unroll
  for (int u = 0; u < 16; u += 2) mul2(z[u], z[u + 1], t[u], t[u + 1], t[u], t[u + 1]);
#pragma unroll
  for (int u = 0; u < 16; u += 2) fma2(y[u], y[u + 1], z[u], z[u + 1], p.c[4], p.c[4], p.c[3], p.c[3]);
#pragma unroll
  for (int i = 2; i >= 0; --i)
#pragma unroll
    for (int u = 0; u < 16; u += 2) fma2(y[u], y[u + 1], y[u], y[u + 1], z[u], z[u + 1], p.c[i], p.c[i]);
#pragma unroll
  for (int u = 0; u < 16; u += 2) mul2(t[u], t[u + 1], t[u], t[u + 1], y[u], y[u + 1]);
}
// Eight products to cap tanh(s / cap) + off + line(u) by the polynomial, in four steps.
template <typename L>
__device__ __forceinline__ void cap_step(const CapPoly& p, int part, float (&t)[8], float (&z)[8], float (&y)[8], L line,
                                         bool lined, float off) {
  // (each operation over the four pairs before the next)
  if (part == 0) {
#pragma unroll
    for (int u = 0; u < 8; u += 2) mul2(z[u], z[u + 1], t[u], t[u + 1], t[u], t[u + 1]);
#pragma unroll
    for (int u = 0; u < 8; u += 2) fma2(y[u], y[u + 1], z[u], z[u + 1], p.c[4], p.c[4], p.c[3], p.c[3]);
  } else if (part == 1) {
#pragma unroll
    for (int u = 0; u < 8; u += 2) fma2(y[u], y[u + 1], y[u], y[u + 1], z[u], z[u + 1], p.c[2], p.c[2]);
  } else if (part == 2) {
#pragma unroll
    for (int u = 0; u < 8; u += 2) fma2(y[u], y[u + 1], y[u], y[u + 1], z[u], z[u + 1], p.c[1], p.c[1]);
  } else {
#pragma unroll
    for (int u = 0; u < 8; u += 2) fma2(y[u], y[u + 1], y[u], y[u + 1], z[u], z[u + 1], p.c[0], p.c[0]);
#pragma unroll
    for (int u = 0; u < 8; u += 2) {
      float f0 = off, f1 = off;
      if (lined) add2(f0, f1, line(u), line(u + 1), off, off);
      fma2(t[u], t[u + 1], t[u], t[u + 1], y[u], y[u + 1], f0, f1);
    }
  }
}
// 16 columns of tensor memory into r[OFF ..] and their largest value.
template <int OFF>
__device__ __forceinline__ void ld16_max(uint32_t taddr, uint32_t (&r)[32], float& m) {
  asm volatile(
      "tcgen05.ld.red.sync.aligned.32x32b.x16.max.f32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, %16, [%17];"
      : "=r"(r[OFF + 0]), "=r"(r[OFF + 1]), "=r"(r[OFF + 2]), "=r"(r[OFF + 3]), "=r"(r[OFF + 4]),
        "=r"(r[OFF + 5]), "=r"(r[OFF + 6]), "=r"(r[OFF + 7]), "=r"(r[OFF + 8]), "=r"(r[OFF + 9]),
        "=r"(r[OFF + 10]), "=r"(r[OFF + 11]), "=r"(r[OFF + 12]), "=r"(r[OFF + 13]),
        "=r"(r[OFF + 14]), "=r"(r[OFF + 15]), "=f"(m)
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void wait_ld_max(float (&m)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(m[0]), "+f"(m[1]), "+f"(m[2]), "+f"(m[3]), "+f"(m[4]), "+f"(m[5]), "+f"(m[6]), "+f"(m[7])
               :
               : "memory");
}

// 8 columns of tensor memory, waited for.
__device__ __forceinline__ void ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr)
      : "memory");
}
// 32 columns of tensor memory and their largest value (both valid after a tcgen05.wait::ld).
__device__ __forceinline__ void ld32_max(uint32_t taddr, uint32_t (&r)[32], float& m) {
  asm volatile(
      "tcgen05.ld.red.sync.aligned.32x32b.x32.max.f32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, %32, [%33];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=f"(m)
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void wait_ld_max(float (&m)[4]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : "+f"(m[0]), "+f"(m[1]), "+f"(m[2]), "+f"(m[3]) : : "memory");
}

// ---- barriers and MMAs by shared-window address. Waits end as those of the shared header do: when the phase
// completes, when another role has given up (abort flag, where given), or after two seconds.
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(1000u)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool bar_test(uint32_t bar, uint32_t parity) {
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
__device__ __forceinline__ uint32_t timer_lo() {
  uint32_t t;
  asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
  return t;
}
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, uint32_t abort_at) {
  if (bar_test(bar, parity)) return true;  // (most phases are complete by then; 1 to 3% faster than a suspending probe)
  const uint32_t t0 = timer_lo();
  for (uint32_t it = 1; it < (1u << 30); ++it) {
    if (bar_try(bar, parity)) return true;
    if ((it & 63u) == 0) {
      uint32_t gone = 0;
      if (abort_at) asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(gone) : "r"(abort_at) : "memory");
      if (gone) return false;
      if (timer_lo() - t0 > (uint32_t)kWaitTimeoutNs) break;
    }
  }
  if (abort_at) asm volatile("st.volatile.shared.u32 [%0], 1;" ::"r"(abort_at) : "memory");
  return false;
}
// The same by a whole warp, which goes on together and with one answer.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint32_t abort_at) {
  return __all_sync(0xffffffffu, bar_wait(bar, parity, abort_at));
}
__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}
// Upper halves of the operand descriptors (128-byte swizzle, version 1, 1024 bytes between groups of eight
// rows); lower halves: the address / 16, and for V, read as an MN-major operand, the distance between
// its blocks of 64 channels (16384 bytes) in the leading-offset field.
constexpr uint32_t kDescHi = (2u << 29) | (1u << 14) | (1024u >> 4);
constexpr uint32_t kLboK = 1u << 16, kLboV = (16384u >> 4) << 16;
// One elected lane of a converged warp issues; `acc` 0: D is overwritten.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
      "r"(a_lo | kLboK), "r"(b_lo | kLboK), "r"(idesc), "r"(acc), "n"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 db;\n\t"
      "mov.b64 db, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d),
      "r"(a_tmem), "r"(b_lo | kLboV), "r"(idesc), "r"(acc), "n"(kDescHi)
      : "memory");
}
// Arrives on the barrier when every MMA issued by the elected thread so far is done.
__device__ __forceinline__ void commit_to(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
      : "memory");
}

// Key tile (after the CTA's first) of step j. With a bias the scores fall with the distance on either side: nearest
// tiles first, the first `left` steps to the left, the others to the right, so that the maximum is met at
// once. (In ascending order a steep slope raised it, and rescaled O, at every tile: 8K causal 479 us
// against 437.)
__device__ __forceinline__ int tile_of(int j, int left) { return j < left ? left - 1 - j : j; }

// O of a row times alpha, in tensor memory.
template <int DP>
__device__ __forceinline__ void rescale_o(uint32_t tO, float alpha) {
#pragma unroll 1
  for (int c = 0; c < DP / 32; ++c) {
    uint32_t o[32];
    tmem_ld32(tO + c * 32, o);
    tmem_wait_ld(o);
#pragma unroll
    for (int u = 0; u < 32; u += 2) {
      float f0, f1;
      mul2(f0, f1, __uint_as_float(o[u]), __uint_as_float(o[u + 1]), alpha, alpha);
      o[u] = __float_as_uint(f0);
      o[u + 1] = __float_as_uint(f1);
    }
    tmem_st32(tO + c * 32, o);
  }
}

// What the roles of a CTA agree on, as words of shared memory: each role loads what it uses (kept in
// registers across the split they spilled, and with the shared memory taken a spill is an L2 access).
enum Word : uint32_t {
  kWTmem = 0, kWAbort = 4, kWJ0 = 16, kWTiles = 20, kWTilesA = 24, kWPrefix = 28, kWRed = 32,
  kWSeq = 48, kWSplit = 52, kWLeft = 56, kWSeen = 60, kWClean = 64
};
__device__ __forceinline__ int lds(uint32_t at) {
  int v;
  asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void sts(uint32_t at, int v) {
  asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}

// CAP / BIAS: the score modification that is compiled in; the masks are a matter of each tile.
template <int DP, bool BF16, bool CAP, bool BIAS>
__global__ void __launch_bounds__(Cfg<DP>::kThreads, Cfg<DP>::kPerSm)
    scored_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, const ScoredArgs a) {
  using C = Cfg<DP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  // shared-window addresses: operands, barriers, abort flag (32 bits each: the control warps have few registers)
  const uint32_t sbase = smem_u32(sm), sK = sbase + C::kOffK, sV = sbase + C::kOffV;
  const uint32_t q_full = sbase + C::kOffBar;
  const uint32_t k_full = q_full + 8, k_empty = k_full + 8 * C::kKStages;
  const uint32_t v_full = k_empty + 8 * C::kKStages, v_empty = v_full + 8 * C::kVStages;
  const uint32_t v_clean = v_empty + 8 * C::kVStages;  // V without what padding held
  const uint32_t s_full = v_clean + 8 * C::kVStages;   // [2] scores of a tile are in tensor memory
  const uint32_t s_free = s_full + 16;                 // [2] and in registers (P beside S)
  const uint32_t p_half = s_free + 16;                 // [2] P of the first 64 keys is written (P over S)
  const uint32_t p_full = p_half + 16;                 // [2] all of P is
  const uint32_t o_full = p_full + 16;                 // [2] P V is done
  const uint32_t drain = o_full + 16;                  // [2]
  const uint32_t misc = sbase + C::kOffMisc, abort_at = misc + kWAbort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the work item: head, sequence, key split, pair of query tiles (those with the most keys first when causal)
  const int q0 = (a.causal ? (int)(gridDim.y - 1 - blockIdx.y) : (int)blockIdx.y) * C::kRows;
  const int hk = (int)blockIdx.x / a.ctas_kv, h_at = ((int)blockIdx.x - hk * a.ctas_kv) * a.heads;
  const int h0 = hk * (a.hq / a.hkv) + h_at, nh = min(a.heads, a.hq / a.hkv - h_at);  // its heads
  const bool has_b = C::kTiles == 2 && (nh > a.per_tile || a.nq - q0 > 128);

  if (threadIdx.x == 0) {
    bar_init(q_full, 1);
    for (int i = 0; i < C::kKStages; ++i) { bar_init(k_full + 8 * i, 1); bar_init(k_empty + 8 * i, 1); }
    for (int i = 0; i < C::kVStages; ++i) {
      bar_init(v_full + 8 * i, 1);
      bar_init(v_empty + 8 * i, 1);
      bar_init(v_clean + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(s_full + 8 * i, 1);
      bar_init(s_free + 8 * i, 128);
      bar_init(p_half + 8 * i, 128);
      bar_init(p_full + 8 * i, 128);
      bar_init(o_full + 8 * i, 1);
      bar_init(drain + 8 * i, 1);
    }
    sts(abort_at, 0);
    // smallest and largest id of the rows, first and last key tile with such ids
    sts(misc + kWRed, INT32_MAX);
    sts(misc + kWRed + 4, -1);
    sts(misc + kWRed + 8, INT32_MAX);
    sts(misc + kWRed + 12, -1);
    fence_mbar_init();
  }
  if (warp == C::kCtl + 1) {
    tmem_alloc(reinterpret_cast<uint32_t*>(sm + C::kOffMisc + kWTmem), C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  // the status word: nothing but a wait of two seconds can set it after this
  if (a.err && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0) *a.err = 0;

  // Q is on its way while the key tiles are found
  if (warp == C::kCtl && lane == 0) {
    tma_prefetch_desc(&tmQ);
    const int b = (int)blockIdx.z / a.splits;
    bar_expect(q_full, (has_b ? 2 : 1) * C::kQBytes);
    if (a.heads == 1) {
      for (int t = 0; t < (has_b ? 2 : 1); ++t)
        for (int c = 0; c < C::kChunks; ++c)
          tma_4d(sbase + t * C::kQBytes + c * 16384, &tmQ, q_full, c * 64, q0 + t * 128, h0, b);
    } else {
      // (the rows of heads that are not there come from behind the last head: zeros)
      for (int i = 0; i < (has_b ? 2 : 1) * a.per_tile; ++i)
        for (int c = 0; c < C::kChunks; ++c)
          tma_4d(sbase + i / a.per_tile * C::kQBytes + c * 16384 + (((i % a.per_tile) * 128) << a.row_bits), &tmQ, q_full,
                 c * 64, 0, i < nh ? h0 + i : a.hq, b);
    }
  }

  // ---- the key tiles of this CTA
  // keys that a row sees at most
  auto limit_of = [&](int row, int prefix) -> int {
    if (!a.causal) return a.nk;
    long long n = (long long)row + a.q_offset + 1;
    n = n > prefix ? n : prefix;
    return (int)(n < 0 ? 0 : n < a.nk ? n : a.nk);
  };
  {
    const int b = (int)blockIdx.z / a.splits, split = (int)blockIdx.z - b * a.splits;
    const int rows = min(C::kRows, a.nq - q0), prefix = a.prefix ? __ldg(&a.prefix[b]) : 0;
    const int seen = limit_of(q0 + rows - 1, prefix);  // (what the last row sees, the rows before it see in part)
    int lo = 0, hi = (seen + 127) / 128;
    const int hi_a = (limit_of(q0 + min(rows, 128) - 1, prefix) + 127) / 128;
    if (a.doc_q) {
      int* red = reinterpret_cast<int*>(sm + C::kOffMisc + kWRed);
      if (warp < C::kCtl) {
        const int id = (int)threadIdx.x < rows ? __ldg(&a.doc_q[(int64_t)b * a.nq + q0 + threadIdx.x]) : -1;
        const int most = __reduce_max_sync(0xffffffffu, id);
        const int least = (int)__reduce_min_sync(0xffffffffu, (unsigned)id);  // (negative ids come last)
        if (lane == 0 && most >= 0) { atomicMin(&red[0], least); atomicMax(&red[1], most); }
      }
      __syncthreads();
      const int dlo = red[0], dhi = red[1];
      for (int j = threadIdx.x; j < hi; j += C::kThreads) {
        const DocTile t = a.doc_tiles[(int64_t)b * a.k_tiles + j];
        if (t.lo <= t.hi && t.hi >= dlo && t.lo <= dhi) { atomicMin(&red[2], j); atomicMax(&red[3], j); }
      }
      __syncthreads();
      lo = min(red[2], hi);
      hi = min(hi, red[3] + 1);
    }
    if (hi < lo) hi = lo;
    if (a.splits > 1) {
      const int n = hi - lo;
      hi = lo + (int)((long long)n * (split + 1) / a.splits);
      lo += (int)((long long)n * split / a.splits);
    }
    if (threadIdx.x == 0) {
      sts(misc + kWJ0, lo);
      sts(misc + kWTiles, hi - lo);
      // tile A leaves out the last key tile where that lies behind all of its rows (unless it comes first)
      sts(misc + kWTilesA, has_b && !BIAS ? max(0, min(hi, max(hi_a, hi - 1)) - lo) : hi - lo);
      // with a bias, the tiles up to the rows' own position come first, from there to the left
      const long long at = ((long long)q0 + rows - 1 + a.q_offset) / 128;
      sts(misc + kWLeft, BIAS ? (int)max(0LL, min(at + 1 - lo, (long long)(hi - lo))) : 0);
      sts(misc + kWPrefix, prefix);
      sts(misc + kWSeq, b);
      // V rows that no row of this CTA sees may hold anything: padding, and what lies behind the last key seen
      sts(misc + kWSeen, seen);
      sts(misc + kWClean, a.doc_k != nullptr || (seen < a.nk && seen < hi * 128));
      sts(misc + kWSplit, split);
    }
  }
  __syncthreads();

  if (warp >= C::kCtl) {
    regs_dec<C::kRegsCtl>();
    if (warp == C::kCtl) {
      // ========================================================= TMA producer
      const int n_tiles = lds(misc + kWTiles), row0 = lds(misc + kWJ0) * 128, b = lds(misc + kWSeq);
      const int left = lds(misc + kWLeft);
      if (lane == 0 && n_tiles == 0) bar_wait(q_full, 0, 0);  // (Q lands before the shared memory goes away)
      if (lane == 0 && n_tiles > 0) {
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
        int nk = 0, nv = 0;
        bool ok = true;
        for (int j = 0; j < n_tiles; ++j) {
          const int sk = j % C::kKStages, sv = j % C::kVStages, row = row0 + tile_of(j, left) * 128;
          if (j >= C::kKStages) ok = bar_wait(k_empty + 8 * sk, ((j / C::kKStages) - 1) & 1, abort_at);
          if (!ok) break;
          bar_expect(k_full + 8 * sk, C::kKBytes);
          for (int c = 0; c < C::kChunks; ++c)
            tma_4d(sK + sk * C::kKBytes + c * 16384, &tmK, k_full + 8 * sk, c * 64, row, hk, b);
          ++nk;
          if (j >= C::kVStages) ok = bar_wait(v_empty + 8 * sv, ((j / C::kVStages) - 1) & 1, abort_at);
          if (!ok) break;
          bar_expect(v_full + 8 * sv, C::kVBytes);
          for (int c = 0; c < C::kChunks; ++c)
            tma_4d(sV + sv * C::kVBytes + c * 16384, &tmV, v_full + 8 * sv, c * 64, row, hk, b);
          ++nv;
        }
        if (!ok) {
          // copies in flight land before the shared memory goes away (abort address 0: no one cuts this short)
          bar_wait(q_full, 0, 0);
          for (int j = max(0, nk - C::kKStages); j < nk; ++j)
            bar_wait(k_full + 8 * (j % C::kKStages), (j / C::kKStages) & 1, 0);
          for (int j = max(0, nv - C::kVStages); j < nv; ++j)
            bar_wait(v_full + 8 * (j % C::kVStages), (j / C::kVStages) & 1, 0);
          if (a.err) record_error(a.err, kDevTimeout);
        }
      }
    } else if (warp == C::kCtl + 3) {
      // ================================== V rows of padding and behind the last key seen become zero
      if (lds(misc + kWClean)) {
        const int n_tiles = lds(misc + kWTiles), j0 = lds(misc + kWJ0), b = lds(misc + kWSeq);
        const int left = lds(misc + kWLeft), seen = lds(misc + kWSeen);
        bool ok = true;
        for (int j = 0; j < n_tiles && ok; ++j) {
          const int sv = j % C::kVStages;
          ok = warp_wait(v_full + 8 * sv, (j / C::kVStages) & 1, abort_at);
          if (!ok) break;
          const int tile = j0 + tile_of(j, left);
          const bool pad = a.doc_k && a.doc_tiles[(int64_t)b * a.k_tiles + tile].pad;
          if (pad || seen < min(a.nk, tile * 128 + 128)) {
            for (int i = 0; i < 4; ++i) {
              const int row = i * 32 + lane, key = tile * 128 + row;
              if (key < a.nk && (key >= seen || (pad && __ldg(&a.doc_k[(int64_t)b * a.nk + key]) < 0)))
                for (int c = 0; c < C::kChunks; ++c)
                  for (int u = 0; u < 8; ++u)
                    *reinterpret_cast<uint4*>(sm + C::kOffV + sv * C::kVBytes + c * 16384 + row * 128 + u * 16) =
                        make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
          }
          __syncwarp();
          if (lane == 0) bar_arrive(v_clean + 8 * sv);
        }
        if (!ok && lane == 0 && a.err) record_error(a.err, kDevTimeout);
      }
    } else if (warp == C::kCtl + 1) {
      // ========================================================= MMA issuers
      const int n_tiles = lds(misc + kWTiles), n_a = lds(misc + kWTilesA);
      const uint32_t tmem = lds(misc + kWTmem);
      const uint32_t fmt = BF16 ? 1 : 0;
      const uint32_t id_qk = make_idesc(1, fmt, fmt, 128, 128), id_pv = make_idesc(1, fmt, fmt, 128, DP) | kIdescTransB;
      const uint32_t v_in = lds(misc + kWClean) ? v_clean : v_full;
      // scores of query tile x against key tile j into S buffer sb
      auto issue_qk = [&](int x, int j, int sb) {
        const uint32_t st = (uint32_t)j % C::kKStages;
        if (!warp_wait(k_full + 8 * st, (j / C::kKStages) & 1, abort_at)) return false;
        tc_fence_after();
        const uint32_t qx = (sbase + x * C::kQBytes) >> 4, kx = (sK + st * C::kKBytes) >> 4;
#pragma unroll
        for (int k = 0; k < DP / 16; ++k) {
          constexpr uint32_t kStep = 16384 >> 4;
          const uint32_t off = (k >> 2) * kStep + (k & 3) * 2;
          mma_ss(tmem + sb * 128, qx + off, kx + off, id_qk, k > 0);
        }
        commit_to(s_full + 8 * sb);
        return true;
      };
      // O of query tile x += P V of key tile j
      auto issue_pv = [&](int x, int j, uint32_t p_col, bool done) {
        const uint32_t sv = (uint32_t)j % C::kVStages;
        if (!warp_wait(v_in + 8 * sv, (j / C::kVStages) & 1, abort_at)) return false;
        if (!warp_wait((C::kOver ? p_half : p_full) + 8 * x, j & 1, abort_at)) return false;
        tc_fence_after();
        const uint32_t d_o = tmem + C::kTmemO + x * DP, a_p = tmem + p_col;
        const uint32_t vx = (sV + sv * C::kVBytes) >> 4;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (C::kOver && k == 4) {
            if (!warp_wait(p_full + 8 * x, j & 1, abort_at)) return false;
            tc_fence_after();
          }
          mma_ts(d_o, a_p + k * 8, vx + (k * 2048 >> 4), id_pv, (j > 0 || k > 0) ? 1u : 0u);
        }
        if (done) commit_to(o_full + 8 * x);
        return true;
      };
      bool ok = n_tiles == 0 || warp_wait(q_full, 0, abort_at);
      if constexpr (C::kOver) {
        // One issuer, the tiles in turn, P V and the next scores of one tile together: the tiles then stay
        // half a period apart, one in its softmax while the other has the tensor core. (An issuer per
        // tile lets them fall into step, both in the softmax and then both waiting: 1.2 times slower.)
        // Each item has one commit, of its scores, which also tells that P V before them is done: a
        // second commit in a row holds the issuer up by some 300 cycles, so the softmax releases
        // the K and V stages. A single query tile has both S buffers and its scores a tile earlier.
        const int nx = has_b ? 2 : 1, lead = has_b ? 1 : 2;
#pragma unroll 1
        for (int j = -lead; j < n_tiles && ok; ++j)
#pragma unroll 1
          for (int x = 0; x < nx && ok; ++x) {
            const int n = x == 0 ? n_a : n_tiles, sb = nx == 2 ? x : j & 1;
            if (j >= 0 && j < n) ok = issue_pv(x, j, sb * 128, nx == 1 || j + 1 == n);
            if (ok && j + lead < n) ok = issue_qk(x, j + lead, sb);
          }
      } else {
        // the next scores as soon as the softmax holds the last ones, then P V
#pragma unroll 1
        for (int j = -1; j < n_tiles && ok; ++j) {
          if (j >= 0 && j + 1 < n_tiles) ok = warp_wait(s_free, j & 1, abort_at);
          if (ok && j + 1 < n_tiles) ok = issue_qk(0, j + 1, 0);
          if (ok && j >= 0) ok = issue_pv(0, j, C::kTmemP, true);
        }
      }
      // every MMA has finished before tensor memory is released
      commit_to(drain);
      warp_wait(drain, 0, 0);
      __syncwarp();
      if (!ok && lane == 0 && a.err) record_error(a.err, kDevTimeout);
    }
  } else {
    regs_inc<C::kRegsSoft>();
    // =========================================================== softmax of tile x
    const int x = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int head = a.heads == 1 ? 0 : x * a.per_tile + (r >> a.row_bits);  // of this CTA's
    const int row = a.heads == 1 ? q0 + x * 128 + r : r & ((1 << a.row_bits) - 1);
    const bool active = x == 0 || has_b, valid = active && row < a.nq && head < nh;
    // head_dim 128 and one query tile: the scores alternate between both S buffers, P V of the tile
    // before is waited for at each tile
    const bool solo = C::kOver && !has_b;
    const bool releases = (threadIdx.x & 127) == 0 && (!C::kOver || x == 1 || solo);
    const uint32_t tmem = lds(misc + kWTmem);
    const int j0 = lds(misc + kWJ0), prefix = lds(misc + kWPrefix), b = lds(misc + kWSeq), h = h0 + (valid ? head : 0);
    const uint32_t tO = tmem + lane_base + C::kTmemO + x * DP;
    const int my_tiles = lds(misc + (x == 0 ? kWTilesA : kWTiles)), left = lds(misc + kWLeft);
    const int limit = valid ? limit_of(row, prefix) : 0;
    // (any negative id is padding: -1, apart from the -2 of a tile of several documents)
    const int dq = !a.doc_q ? 0 : valid ? max(__ldg(&a.doc_q[(int64_t)b * a.nq + row]), -1) : -1;
    const int pos = row + a.q_offset;
    constexpr float kSlack = BF16 ? 60.0f : 7.0f;  // by how much a maximum may be overestimated
    float slope = 0.f;
    if constexpr (BIAS) slope = __ldg(&a.slopes[h]) * kL2e;
    // (a warp's rows may be of heads with different slopes; where fp16's few bits of slack make many slopes steep, their
    // maximum is taken exactly: 8192 causal with slopes of 0.5 455 us, with gentle ones 407; with a cap it would cost a
    // capped score more per key, and steep slopes take the loop)
    constexpr bool kExact = !BF16 && !CAP;
    const bool gentle = !BIAS || __all_sync(0xffffffffu, fabsf(slope) * 15.0f <= kSlack);
    const float cap_m2 = -2.0f * a.cap2, cap_in = a.cap_k;
    // fp16 weights are held at up to 2^(7 + 8): 7 bits more before the smallest lose bits
    constexpr float kHead = BF16 ? 0.f : 7.0f;
    float m = kNegInf;                             // the frame, base 2
    float l = 0.f;
    bool ok = true;
    // the document that a tile's keys are all of, or -2; read a step ahead
    auto only_of = [&](int j) {
      const DocTile t = a.doc_tiles[(int64_t)b * a.k_tiles + j0 + (BIAS ? tile_of(j, left) : j)];
      return t.mixed ? -2 : t.lo;
    };
    int only = a.doc_k && my_tiles > 0 ? only_of(0) : 0, only_next = 0;
    if (active) {
      for (int j = 0; j < my_tiles && ok; ++j, only = only_next) {
        if (a.doc_k && j + 1 < my_tiles) only_next = only_of(j + 1);
        const int sb = solo ? j & 1 : x;
        const uint32_t tS = tmem + lane_base + sb * 128, tP = C::kOver ? tS : tmem + lane_base + C::kTmemP;
        const int tile = j0 + (BIAS ? tile_of(j, left) : j), kv0 = tile * 128;
        // ---- does every row of the warp see every key of the tile?
        bool whole = limit - kv0 >= 128;
        if (a.doc_k) whole = whole && only == dq;
        whole = whole || !valid;  // (rows behind the last one are not written)
        // The bias along a tile that lies on one side of every row's position is base + step u. Its largest value
        // beside the largest product of each 16 keys bounds the maximum by at most 15 steps too much, which the
        // frame's headroom takes where they are few.
        bool fast = __all_sync(0xffffffffu, whole);
        float mul = a.c2, step = 0.f, base = 0.f;
        const float dist = static_cast<float>(pos - kv0);  // exact below 2^24
        if constexpr (BIAS) {
          const bool all_left = __all_sync(0xffffffffu, kv0 + 127 <= pos);
          fast = fast && (gentle || kExact) && (all_left || __all_sync(0xffffffffu, kv0 >= pos));
          step = all_left ? slope : -slope;
          base = -step * dist;
        }
        ok = warp_wait(s_full + 8 * sb, (solo ? j >> 1 : j) & 1, abort_at);
        if (!ok) break;
        if (releases) {  // K of this tile has been read, and V of the last (where this barrier tells it)
          bar_arrive(k_empty + 8 * ((uint32_t)j % C::kKStages));
          if (C::kOver && !solo && j > 0) bar_arrive(v_empty + 8 * ((uint32_t)(j - 1) % C::kVStages));
        }
        tc_fence_after();
        float t_max = kNegInf, m_use = 0.f;
        float g0 = 0.f, g1 = 0.f, g2 = 0.f, g3 = 0.f;
        uint32_t s[4][32];
        if (fast) {
          // the products; cap and scale keep their order, so the largest of each 16 or 32 gives the maximum
          float cm[BIAS ? 8 : 4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if constexpr (BIAS) {
              ld16_max<0>(tS + c * 32, s[c], cm[2 * c]);
              ld16_max<16>(tS + c * 32 + 16, s[c], cm[2 * c + 1]);
            } else {
              ld32_max(tS + c * 32, s[c], cm[c]);
            }
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_wait_ld(s[c]);
          wait_ld_max(cm);
          auto capped = [&](float v) {
            return CAP ? fmaf(rcpf(1.0f + ex2f(v * cap_in)), cap_m2, a.cap2) : v * a.c2;
          };
          if constexpr (BIAS) {
            if (gentle || !kExact) {
              const float end = step > 0.f ? 15.0f * step : 0.f;
#pragma unroll
              for (int c = 0; c < 8; ++c) t_max = fmaxf(t_max, fmaf(step, static_cast<float>(c * 16), capped(cm[c])));
              t_max += end;
            } else {  // (steep slopes: the maximum itself)
#pragma unroll
              for (int c = 0; c < 4; ++c) {
#pragma unroll
                for (int u = 0; u < 32; u += 2) {
                  float f0, f1;
                  fma2(f0, f1, __uint_as_float(s[c][u]), __uint_as_float(s[c][u + 1]), a.c2, a.c2,
                       step * static_cast<float>(c * 32 + u), step * static_cast<float>(c * 32 + u + 1));
                  t_max = max3(t_max, f0, f1);
                }
              }
            }
            t_max += base;
          } else {
            t_max = capped(fmaxf(max3(cm[0], cm[1], cm[2]), cm[3]));
          }
          if constexpr (CAP) {
            // every product of the warp within the polynomial's range?
            float big = 0.f;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
#pragma unroll
              for (int u = 0; u < 32; u += 2)
                big = max3(big, fabsf(__uint_as_float(s[c][u])), fabsf(__uint_as_float(s[c][u + 1])));
            }
            fast = __all_sync(0xffffffffu, big <= a.poly.most);
          }
        }
        if (!fast) {
          // 32 or 64 keys at a time, in place: scores (products, where there is neither cap nor bias), masked. A loop, since
          // the CTAs and warps of an SM are seldom in the same place and share the instruction cache: as straight
          // code of 128 keys, plain prompts took 8% longer at head_dim 64. (Capped and biased, 64 keys are longer
          // than 32: packed documents 148 against 141 us; plain shorter, 81 against 88.)
          int id[4] = {-1, -1, -1, -1};
          const bool by_doc = a.doc_k && !__all_sync(0xffffffffu, only == dq || !valid);
          if (by_doc) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int key = kv0 + c * 32 + lane;
              if (key < a.nk) id[c] = __ldg(&a.doc_k[(int64_t)b * a.nk + key]);
            }
          }
          t_max = kNegInf;
          constexpr int kN = CAP || BIAS ? 1 : 2;
#pragma unroll 1
          for (int c = 0; c < 4; c += kN) {
            uint32_t part[kN][32], bits[kN];
#pragma unroll
            for (int i = 0; i < kN; ++i) tmem_ld32(tS + (c + i) * 32, part[i]);
            // which of the keys this row sees, as bits; each document among the warp's rows in turn, its keys by ballot
#pragma unroll
            for (int i = 0; i < kN; ++i) {
              const int k = limit - kv0 - (c + i) * 32;
              bits[i] = k >= 32 ? 0xffffffffu : k <= 0 ? 0u : (1u << k) - 1u;
            }
            if (by_doc) {
              uint32_t todo = __ballot_sync(0xffffffffu, dq >= 0), mine[kN] = {};
              while (todo) {
                const int one = __shfl_sync(0xffffffffu, dq, __ffs(todo) - 1);
                const bool me = dq == one;
#pragma unroll
                for (int i = 0; i < kN; ++i) {
                  const int key_id = c + i == 0 ? id[0] : c + i == 1 ? id[1] : c + i == 2 ? id[2] : id[3];
                  const uint32_t v = __ballot_sync(0xffffffffu, key_id == one);
                  if (me) mine[i] = v;
                }
                todo &= ~__ballot_sync(0xffffffffu, me);
              }
#pragma unroll
              for (int i = 0; i < kN; ++i) bits[i] &= mine[i];
            }
#pragma unroll
            for (int i = 0; i < kN; ++i) tmem_wait_ld(part[i]);
            bool small = false;
            if constexpr (CAP) {
              float b4[4] = {0.f, 0.f, 0.f, 0.f};  // (one chain: documents of head_dim 128 161 us against 157)
#pragma unroll
              for (int u = 0; u < 32; u += 8) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  b4[k] = max3(b4[k], fabsf(__uint_as_float(part[0][u + 2 * k])), fabsf(__uint_as_float(part[0][u + 2 * k + 1])));
              }
              float big = fmaxf(max3(b4[0], b4[1], b4[2]), b4[3]);
              small = __all_sync(0xffffffffu, big <= a.poly.most);
              // A key that no row of the warp sees must not choose the form: then the products that are seen are looked
              // at, from tensor memory. (8 heads x 16383 in 14 documents, d 64: 139 us; by selects for every part 155, in
              // this branch 142; by all products, seen or not, 133. Scores far beyond the cap, 8192 causal, d 128: 951 us;
              // looked at in parts that every row sees too, 1109.)
              if (!small && !__all_sync(0xffffffffu, bits[0] == 0xffffffffu)) {
                big = 0.f;
#pragma unroll 1
                for (int u = 0; u < 32; u += 8) {
                  uint32_t r[8];
                  ld8(tS + c * 32 + u, r);
#pragma unroll
                  for (int k = 0; k < 8; ++k) big = fmaxf(big, bits[0] >> (u + k) & 1u ? fabsf(__uint_as_float(r[k])) : 0.f);
                }
                small = __all_sync(0xffffffffu, big <= a.poly.most);
              }
            }
#pragma unroll
            for (int g = 0; g < 2 * kN; ++g) {
              const int i = g >> 1, at = (g & 1) * 16;
              float t[16];
#pragma unroll
              for (int u = 0; u < 16; ++u) t[u] = __uint_as_float(part[i][at + u]);
              if constexpr (CAP) {
                if (small) cap_polynomial(t, a.poly);
                else cap_quotient(t, cap_in, cap_m2, a.cap2);
              }
              if constexpr (BIAS) {
                const float d0 = dist - static_cast<float>(c * 32 + g * 16);
#pragma unroll
                for (int u = 0; u < 16; u += 2) {
                  const float b0 = -slope * fabsf(d0 - static_cast<float>(u)), b1 = -slope * fabsf(d0 - static_cast<float>(u + 1));
                  if constexpr (CAP) add2(t[u], t[u + 1], t[u], t[u + 1], b0, b1);
                  else fma2(t[u], t[u + 1], t[u], t[u + 1], a.c2, a.c2, b0, b1);
                }
              }
#pragma unroll
              for (int u = 0; u < 16; ++u) {
                t[u] = bits[i] >> (at + u) & 1u ? t[u] : kNegInf;
                part[i][at + u] = __float_as_uint(t[u]);
              }
#pragma unroll
              for (int u = 0; u < 16; u += 2) t_max = max3(t_max, t[u], t[u + 1]);
            }
#pragma unroll
            for (int i = 0; i < kN; ++i) tmem_st32(tS + (c + i) * 32, part[i]);
          }
          tmem_wait_st();
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(tS + c * 32, s[c]);
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_wait_ld(s[c]);
          mul = CAP || BIAS ? 1.0f : a.c2;
          t_max *= CAP || BIAS ? 1.0f : a.c2;
          step = base = 0.f;
        }
        if constexpr (!C::kOver) {  // S is in registers
          tc_fence_before();
          bar_arrive(s_free + 8 * x);
        }
        // P V of the tile before is done: O may be rescaled, P overwritten (it also keeps p_full at most one
        // phase ahead of its issuer). Two tiles at head_dim 128 know it from the scores' barrier.
        auto wait_pv = [&]() {
          if (j > 0 && (!C::kOver || solo)) {
            ok = warp_wait(o_full + 8 * x, (j - 1) & 1, abort_at);
            if (ok) tc_fence_after();
          }
        };
        // The frame m lies kHead below the maximum that set it, and is kept unless that grew by more than 8.
        {
          t_max -= kHead;
          const bool grow = t_max > m + 8.0f || (m == kNegInf && t_max > kNegInf);
          if (__any_sync(0xffffffffu, grow)) {
            const float alpha = grow ? ex2f(m - t_max) : 1.0f;
            m = grow ? t_max : m;
            l *= alpha;
            if (j > 0) {
              wait_pv();
              if (ok) rescale_o<DP>(tO, alpha);
            }
          }
          m_use = m == kNegInf ? 0.f : m;
        }
        if (!ok) break;
        // P = 2^(t - m), summed in 32 bits, rounded once to the operands' type; t is mul s, or with POLY s capped by
        // the polynomial, and LINE adds a bias of base + step u. Eight keys enter per round; a pair's arithmetic, its
        // exponentials and its sum and rounding lie one round apart and are issued in turn, so that the
        // special-function unit (four cycles per exponential and warp) never waits for the others.
        auto weights = [&](auto poly, auto line) {
          constexpr bool POLY = decltype(poly)::value, LINE = decltype(line)::value;
          const float off = base - m_use;
          float st[LINE ? 8 : 1];
          if constexpr (LINE) {
#pragma unroll
            for (int u = 0; u < 8; ++u) st[u] = step * static_cast<float>(u);
          }
          float r0[8], r1[8];  // rounds in flight, the newest first
#pragma unroll
          for (int q = 0; q < 18; ++q) {
            float in[8], mid[8], z[8], y[8], o8 = off;
            if constexpr (LINE) o8 = fmaf(step, static_cast<float>(q * 8), off);
            if (q < 16) {
#pragma unroll
              for (int u = 0; u < 8; ++u) in[u] = __uint_as_float(s[q >> 2][(q & 3) * 8 + u]);
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) mid[u] = r0[u];
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
              // exponentials of the round before
              if (q >= 1 && q < 17) {
                mid[i] = ex2f(mid[i]);
                mid[i + 1] = ex2f(mid[i + 1]);
              }
              // arithmetic of the new round
              if (q < 16) {
                if constexpr (POLY) {
                  cap_step(a.poly, i / 2, in, z, y, [&](int u) { return LINE ? st[u] : 0.f; }, LINE, o8);
                } else {
                  float f0 = o8, f1 = o8;
                  if constexpr (LINE) add2(f0, f1, st[i], st[i + 1], o8, o8);
                  fma2(in[i], in[i + 1], in[i], in[i + 1], mul, mul, f0, f1);
                }
              }
              // sum and rounding of the oldest round
              if (q >= 2) {
                if (i & 2) add2(g2, g3, g2, g3, r1[i], r1[i + 1]);
                else add2(g0, g1, g0, g1, r1[i], r1[i + 1]);
                const int w = (q - 2) * 4 + i / 2;
                s[w >> 5][w & 31] = pack16<BF16>(r1[i], r1[i + 1]);
              }
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              r1[u] = mid[u];
              r0[u] = in[u];
            }
            if (q == 9) {
              wait_pv();
              if (!ok) return;
              if (releases && j > 0 && (!C::kOver || solo)) bar_arrive(v_empty + 8 * ((uint32_t)(j - 1) % C::kVStages));
              tmem_st32(tP, s[0]);
              if (C::kOver) {
                tmem_wait_st();
                tc_fence_before();
                bar_arrive(p_half + 8 * x);
              }
            }
            if (q == 17) tmem_st32(tP + 32, s[1]);
          }
        };
        if constexpr (CAP) {
          if (fast) weights(std::true_type{}, std::integral_constant<bool, BIAS>{});
          else weights(std::false_type{}, std::false_type{});
        } else {
          weights(std::false_type{}, std::integral_constant<bool, BIAS>{});
        }
        if (!ok) break;
        l += (g0 + g1) + (g2 + g3);
        tmem_wait_st();
        tc_fence_before();
        bar_arrive(p_full + 8 * x);
      }
      // ---- out = O / l and the log-sum-exp; a split writes O and its frame to the workspace
      if (ok && my_tiles > 0) {
        // (two tiles at head_dim 128 commit it once, after their last P V)
        const int last = C::kOver && !solo ? 0 : my_tiles - 1;
        ok = warp_wait(o_full + 8 * x, last & 1, abort_at);
        tc_fence_after();
      }
      if (ok) {
        const int b = lds(misc + kWSeq), split = lds(misc + kWSplit);
        const int64_t line = ((int64_t)b * a.hq + h) * a.nq + row;
        const bool seen = my_tiles > 0 && l != 0.f;
        const float inv = seen ? 1.0f / l : 0.f;
        uint16_t* const dst = static_cast<uint16_t*>(a.o) + b * a.o_sb + h * a.o_sh + row * a.o_sn;
        float* const part = a.part_o + ((int64_t)split * a.batch * a.hq * a.nq + line) * DP;
#pragma unroll 1
        for (int c = 0; c < DP / 32 && c * 32 < a.d; ++c) {
          uint32_t o[32];
          if (my_tiles > 0) {
            tmem_ld32(tO + c * 32, o);
            tmem_wait_ld(o);
          }
          if (!seen) {
#pragma unroll
            for (int u = 0; u < 32; ++u) o[u] = 0u;
          }
          if (valid && a.splits > 1) {
#pragma unroll
            for (int u = 0; u < 32; u += 4)
              *reinterpret_cast<uint4*>(part + c * 32 + u) = make_uint4(o[u], o[u + 1], o[u + 2], o[u + 3]);
          } else if (valid && a.vec) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (c * 32 + q * 8 < a.d) {
                uint4 v;
                const float* f = reinterpret_cast<const float*>(o) + q * 8;
                v.x = pack16<BF16>(f[0] * inv, f[1] * inv);
                v.y = pack16<BF16>(f[2] * inv, f[3] * inv);
                v.z = pack16<BF16>(f[4] * inv, f[5] * inv);
                v.w = pack16<BF16>(f[6] * inv, f[7] * inv);
                *reinterpret_cast<uint4*>(dst + c * 32 + q * 8) = v;
              }
          } else if (valid) {
#pragma unroll
            for (int u = 0; u < 32; ++u)
              if (c * 32 + u < a.d)
                dst[c * 32 + u] = static_cast<uint16_t>(pack16<BF16>(__uint_as_float(o[u]) * inv, 0.f) & 0xffffu);
          }
        }
        if (valid) {
          if (a.splits > 1)
            *reinterpret_cast<float2*>(a.part_ml + ((int64_t)split * a.batch * a.hq * a.nq + line) * 2) =
                make_float2(seen ? m : kNegInf, seen ? l : 0.f);
          else if (a.lse)
            a.lse[line] = seen ? (m + __log2f(l)) * kL2 : kNegInf;
        }
      }
      if (!ok && a.err) record_error(a.err, kDevTimeout);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == C::kCtl + 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(lds(misc + kWTmem), C::kTmemCols);
  }
}

// The document ids that each tile of 128 keys holds.
__global__ void __launch_bounds__(128) scored_setup_kernel(const ScoredArgs a) {
  __shared__ int s_lo, s_hi, s_pad;
  if (threadIdx.x == 0) { s_lo = INT32_MAX; s_hi = -1; s_pad = 0; }
  __syncthreads();
  const int key = blockIdx.x * 128 + threadIdx.x;
  if (key < a.nk) {
    const int id = __ldg(&a.doc_k[(int64_t)blockIdx.y * a.nk + key]);
    if (id >= 0) { atomicMin(&s_lo, id); atomicMax(&s_hi, id); }
    else s_pad = 1;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    DocTile t;
    t.lo = s_lo; t.hi = s_hi; t.pad = s_pad;
    t.mixed = s_pad || s_lo != s_hi;
    a.doc_tiles[(int64_t)blockIdx.y * a.k_tiles + blockIdx.x] = t;
  }
}

// Splits joined: one warp per row.
template <bool BF16, int DP>
__global__ void __launch_bounds__(128) scored_join_kernel(const ScoredArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t lines = (int64_t)a.batch * a.hq * a.nq, line = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  pdl_wait();
  if (line >= lines) return;
  float m = kNegInf;
  for (int s = 0; s < a.splits; ++s) m = fmaxf(m, a.part_ml[(s * lines + line) * 2]);
  const float u = m == kNegInf ? 0.f : m;
  float l = 0.f, acc[DP / 32];
#pragma unroll
  for (int c = 0; c < DP / 32; ++c) acc[c] = 0.f;
#pragma unroll 4
  for (int s = 0; s < a.splits; ++s) {
    const float2 x = *reinterpret_cast<const float2*>(a.part_ml + (s * lines + line) * 2);
    const float f = ex2f(x.x - u);
    l = fmaf(x.y, f, l);
#pragma unroll
    for (int c = 0; c < DP / 32; ++c)
      if (c * 32 < a.d) acc[c] = fmaf(a.part_o[(s * lines + line) * DP + c * 32 + lane], f, acc[c]);
  }
  const float inv = l != 0.f ? 1.0f / l : 0.f;
  const int64_t bh = line / a.nq;
  const int row = (int)(line - bh * a.nq), b = (int)(bh / a.hq), h = (int)(bh - (int64_t)b * a.hq);
  uint16_t* dst = static_cast<uint16_t*>(a.o) + b * a.o_sb + h * a.o_sh + row * a.o_sn;
#pragma unroll
  for (int c = 0; c < DP / 32; ++c)
    if (c * 32 + lane < a.d) dst[c * 32 + lane] = static_cast<uint16_t>(pack16<BF16>(acc[c] * inv, 0.f) & 0xffffu);
  if (a.lse && lane == 0) a.lse[line] = l != 0.f ? (m + __log2f(l)) * kL2 : kNegInf;
}

// No keys at all: 0 and -inf.
__global__ void __launch_bounds__(128) scored_empty_kernel(const ScoredArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t lines = (int64_t)a.batch * a.hq * a.nq, line = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (a.err && line == 0 && lane == 0) *a.err = 0;
  if (line >= lines) return;
  const int64_t bh = line / a.nq;
  const int row = (int)(line - bh * a.nq), b = (int)(bh / a.hq), h = (int)(bh - (int64_t)b * a.hq);
  for (int c = lane; c < a.d; c += 32)
    static_cast<uint16_t*>(a.o)[b * a.o_sb + h * a.o_sh + row * a.o_sn + c] = 0;
  if (a.lse && lane == 0) a.lse[line] = kNegInf;
}

// Rows that TMA cannot address (odd head_dim or strides, unaligned or broadcast tensors), copied
// once into rows of dp channels: [batch][heads][n][dp], zeros behind d.
struct CopyArgs {
  const uint16_t* src; int64_t sb, sh, sn;
  uint16_t* dst;
  int heads, n, d, dp;
  int64_t lines;
};
__global__ void __launch_bounds__(128) scored_copy_kernel(const CopyArgs a) {
  const int lane = threadIdx.x & 31;
  for (int64_t line = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5); line < a.lines; line += (int64_t)gridDim.x * 4) {
    const int64_t bh = line / a.n;
    const int row = (int)(line - bh * a.n), b = (int)(bh / a.heads), h = (int)(bh - (int64_t)b * a.heads);
    const uint16_t* src = a.src + b * a.sb + h * a.sh + row * a.sn;
    for (int c = lane; c < a.dp; c += 32) a.dst[line * a.dp + c] = c < a.d ? src[c] : (uint16_t)0;
  }
}

// ------------------------------------------------------------------------------------- host
size_t up256(size_t x) { return (x + 255) / 256 * 256; }
struct ScoredLayout {
  size_t tiles, part_o, part_ml, copy[3], total;
  int dp, k_tiles;
  // the work items (see ScoredArgs) and the key splits of each
  int heads, per_tile, row_bits, ctas_kv, splits;
};
// Key splits: where the items leave SMs idle, as many as fill one wave, of at least four key tiles each.
int splits_of(int64_t items, int64_t tiles, int slots) {
  int64_t s = items > 0 ? slots / items : 1;
  if (s > tiles / 4) s = tiles / 4;
  if (s > kMaxSplits) s = kMaxSplits;
  return s < 1 ? 1 : (int)s;
}
// With at most 128 queries the heads of a key/value head can share a CTA and the keys it loads: as blocks of rows of
// one query tile, or of two, whose softmaxes then overlap. A step over one tile alone takes 5/8 of a step over two
// (1.15 and 1.84 us, biased, head_dim 128); a CTA's start and end are worth four steps, and so is the join of
// splits. The shape of the least time is taken.
void plan_items(int batch, int hq, int hkv, int nq, int nk, ScoredLayout* L) {
  const int group = hq / hkv;
  const int64_t tiles = L->k_tiles;
  const int rows = L->dp == 128 ? Cfg<128>::kRows : Cfg<64>::kRows;  // of a CTA
  const int slots = 152 * (L->dp == 128 ? Cfg<128>::kPerSm : Cfg<64>::kPerSm);
  int bits = 3;
  while (bits < 7 && 1 << bits < nq) ++bits;
  int64_t best = -1;
  for (int form = 0; form < (nq <= 128 && group > 1 ? 1 + rows / 128 : 1); ++form) {
    const int per_tile = form == 0 ? 1 : 128 >> bits, room = form == 2 ? 2 * per_tile : per_tile;
    const int heads = form == 0 ? 1 : group < room ? group : room;
    if (form == 1 && heads == 1) continue;
    const int ctas_kv = (group + heads - 1) / heads;
    const int64_t items = (int64_t)batch * hkv * ctas_kv * (((int64_t)nq + rows - 1) / rows);
    const int splits = splits_of(items, tiles, slots);
    const bool two = rows > 128 && (form == 0 ? nq > 128 : heads > per_tile);
    const int64_t waves = (items * splits + slots - 1) / slots;
    const int64_t time = waves * ((tiles + splits - 1) / splits * (two ? 8 : 5) + 20) + (splits > 1 ? 20 : 0);
    if (best < 0 || time < best) {
      best = time;
      L->heads = heads; L->per_tile = per_tile; L->row_bits = form == 0 ? 7 : bits; L->ctas_kv = ctas_kv;
      L->splits = splits;
    }
  }
}
bool scored_layout(int batch, int hq, int hkv, int nq, int nk, int d, bool packed, bool docs, ScoredLayout* L) {
  if (batch < 0 || hq < 1 || hkv < 1 || hq % hkv || nq < 0 || nk < 0 || d < 1 || d > 128) return false;
  L->dp = d <= 64 ? 64 : 128;
  L->k_tiles = (int)(((int64_t)nk + 127) / 128);
  plan_items(batch, hq, hkv, nq, nk, L);
  size_t o = 256;
  auto take = [&](size_t bytes) { const size_t at = o; o += up256(bytes); return at; };
  L->tiles = take(docs ? (size_t)batch * L->k_tiles * sizeof(DocTile) : 0);
  const size_t lines = (size_t)batch * hq * nq;
  L->part_o = take(L->splits > 1 ? L->splits * lines * L->dp * 4 : 0);
  L->part_ml = take(L->splits > 1 ? L->splits * lines * 8 : 0);
  for (int i = 0; i < 3; ++i) {
    const size_t rows = (size_t)batch * (i == 0 ? hq : hkv) * (i == 0 ? nq : nk);
    L->copy[i] = take(packed ? 0 : rows * L->dp * 2);
  }
  L->total = o;
  return true;
}

template <int DP, bool BF16, bool CAP, bool BIAS>
cudaError_t launch_scored_t(const ScoredArgs& a, const CUtensorMap* maps, dim3 grid, cudaStream_t st) {
  static std::atomic<int> limits[64];
  cudaError_t e = raise_smem_limit(scored_kernel<DP, BF16, CAP, BIAS>, Cfg<DP>::kSmem, limits);
  if (e != cudaSuccess) return e;
  return launch_pdl(scored_kernel<DP, BF16, CAP, BIAS>, grid, dim3(Cfg<DP>::kThreads), Cfg<DP>::kSmem, st, maps[0], maps[1],
                    maps[2], a);
}
template <int DP, bool BF16>
cudaError_t launch_scored(const ScoredArgs& a, const CUtensorMap* maps, dim3 grid, cudaStream_t st) {
  const bool cap = a.cap2 > 0.f, bias = a.slopes != nullptr;
  cudaError_t e = cap ? (bias ? launch_scored_t<DP, BF16, true, true>(a, maps, grid, st)
                              : launch_scored_t<DP, BF16, true, false>(a, maps, grid, st))
                      : (bias ? launch_scored_t<DP, BF16, false, true>(a, maps, grid, st)
                              : launch_scored_t<DP, BF16, false, false>(a, maps, grid, st));
  if (e != cudaSuccess || a.splits == 1) return e;
  const int64_t blocks = ((int64_t)a.batch * a.hq * a.nq + 3) / 4;
  return launch_pdl(scored_join_kernel<BF16, DP>, dim3((unsigned)blocks), dim3(128), 0, st, a);
}

struct View {
  const void* p;
  int64_t sb, sh, sn;
  int heads, n;
};

}  // namespace
}  // namespace sage

using namespace sage;

extern "C" {

size_t sage_scored_attn_workspace_size(int batch, int heads_q, int heads_kv, int seqlen_q, int seqlen_k, int head_dim,
                                       int packed) {
  ScoredLayout L;
  return scored_layout(batch, heads_q, heads_kv, seqlen_q, seqlen_k, head_dim, packed & 1, !(packed & 2), &L) ? L.total : 0;
}

int sage_scored_attn(const sage_tensor* q, const sage_tensor* k, const sage_tensor* v, const sage_tensor* out,
                     float* lse, const float* slopes, const int32_t* prefix_lens, const int32_t* doc_q,
                     const int32_t* doc_k, int batch, int heads_q, int heads_kv, int seqlen_q, int seqlen_k,
                     int head_dim, int dtype, int tensor_layout, int is_causal, float sm_scale, float softcap,
                     int q_offset, int return_lse, void* workspace, size_t workspace_bytes, void* stream) {
  if (!q || !k || !v || !out) return SAGE_ERR_INVALID_ARG;
  if (head_dim < 1 || head_dim > 128) return SAGE_ERR_HEAD_DIM;
  if (dtype != SAGE_F16 && dtype != SAGE_BF16) return SAGE_ERR_DTYPE;
  if (tensor_layout != SAGE_HND && tensor_layout != SAGE_NHD) return SAGE_ERR_INVALID_ARG;
  if (batch < 0 || heads_q < 1 || heads_kv < 1 || seqlen_q < 0 || seqlen_k < 0 ||
      !softcap_ok(softcap, sm_scale, head_dim) || (prefix_lens && !is_causal) || (return_lse && !lse && batch > 0 && seqlen_q > 0))
    return SAGE_ERR_INVALID_ARG;
  // (ids of no rows or of no keys have no address)
  if (!doc_q != !doc_k && batch > 0 && seqlen_q > 0 && seqlen_k > 0) return SAGE_ERR_INVALID_ARG;
  if (heads_q % heads_kv) return SAGE_ERR_GQA;
  for (const void* p : {(const void*)lse, (const void*)slopes, (const void*)prefix_lens, (const void*)doc_q, (const void*)doc_k})
    if (reinterpret_cast<uintptr_t>(p) % 4) return SAGE_ERR_INVALID_ARG;
  if (batch == 0 || seqlen_q == 0) return SAGE_OK;
  const sage_tensor* ts[4] = {q, k, v, out};
  View view[4];
  for (int i = 0; i < 4; ++i) {
    const sage_tensor* t = ts[i];
    const bool keys = i == 1 || i == 2;
    if (!t->data && !(keys && seqlen_k == 0)) return SAGE_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(t->data) % 2) return SAGE_ERR_STRIDE;
    for (int s = 0; s < 3; ++s)
      if (t->stride[s] < 0) return SAGE_ERR_STRIDE;
    const int hi = tensor_layout == SAGE_HND ? 1 : 2, ni = tensor_layout == SAGE_HND ? 2 : 1;
    view[i] = {t->data, t->stride[0], t->stride[hi], t->stride[ni], keys ? heads_kv : heads_q, keys ? seqlen_k : seqlen_q};
  }
  ScoredLayout L;
  // rows that TMA addresses: 16-byte aligned, no zero stride of a dimension that is walked
  bool fits[4];
  for (int i = 0; i < 4; ++i) {
    const View& t = view[i];
    bool ok = head_dim % 8 == 0 && reinterpret_cast<uintptr_t>(t.p) % 16 == 0;
    const int64_t str[3] = {t.sb, t.sh, t.sn}, len[3] = {batch, t.heads, t.n};
    for (int s = 0; s < 3; ++s)
      if (len[s] > 1) ok = ok && str[s] > 0 && str[s] % 8 == 0 && str[s] < (1LL << 38);
    fits[i] = ok;
  }
  const bool packed = fits[0] && fits[1] && fits[2];
  if (!scored_layout(batch, heads_q, heads_kv, seqlen_q, seqlen_k, head_dim, packed, doc_k != nullptr, &L)) return SAGE_ERR_INVALID_ARG;
  const int cta_rows = L.dp == 128 ? Cfg<128>::kRows : Cfg<64>::kRows;
  const int64_t blocks_q = ((int64_t)seqlen_q + cta_rows - 1) / cta_rows;
  // (positions, and with slopes distances, that the kernel holds in 32 bits)
  if (seqlen_k > 0x7fffff00 || seqlen_q > 0x7fffff00 || (int64_t)q_offset + seqlen_q > 0x7fffff00 ||
      q_offset < -0x7fffff00 || (slopes && (int64_t)q_offset - seqlen_k < -0x7fffff00) || blocks_q > 65535 ||
      (int64_t)batch * L.splits > 65535 || (int64_t)batch * heads_q * seqlen_q > (1LL << 32))
    return SAGE_ERR_INVALID_ARG;
  // (the status word alone can do without)
  if (workspace ? reinterpret_cast<uintptr_t>(workspace) % 256 || workspace_bytes < L.total : L.total > SAGE_STATUS_BYTES)
    return SAGE_ERR_WORKSPACE;
  if (!sage_device_supported()) return SAGE_ERR_DEVICE;
  char* w = static_cast<char*>(workspace);
  ScoredArgs a{};
  a.batch = batch; a.hq = heads_q; a.hkv = heads_kv; a.nq = seqlen_q; a.nk = seqlen_k; a.d = head_dim;
  a.dtype = dtype; a.causal = is_causal ? 1 : 0; a.splits = L.splits; a.k_tiles = L.k_tiles; a.q_offset = q_offset;
  a.vec = fits[3] ? 1 : 0;
  a.heads = L.heads; a.per_tile = L.per_tile; a.row_bits = L.row_bits; a.ctas_kv = L.ctas_kv;
  const float scale =
      std::isnan(sm_scale) || sm_scale <= 0.f ? (float)(1.0 / std::sqrt((double)head_dim)) : sm_scale;
  a.c2 = std::fmax((float)(scale * 1.4426950408889634), 1.2e-38f);  // (-inf times it is -inf)
  a.cap2 = (float)(softcap * 1.4426950408889634);
  const double tanh_c[5] = {0.9999997019767761, -0.3333034813404083, 0.13282497227191925, -0.050881292670965195,
                            0.013819585554301739};
  const double cap_x = softcap > 0.f ? (double)scale / softcap : 0.0;
  double scaled = softcap * 1.4426950408889634 * cap_x;
  a.poly.most = softcap > 0.f ? (float)(0.7 / cap_x) : -1.f;
  for (int i = 0; i < 5; ++i, scaled *= cap_x * cap_x) {
    const double c = tanh_c[i] * scaled;
    a.poly.c[i] = (float)c;
    // (a coefficient near the ends of fp32's range: the quotient)
    if (!(std::fabs(c) > 1e-37 && std::fabs(c) < 1e30)) a.poly.most = -1.f;
  }
  a.cap_k = softcap > 0.f ? (float)(2.0 * 1.4426950408889634 * scale / softcap) : 0.f;
  a.o = out->data; a.o_sb = view[3].sb; a.o_sh = view[3].sh; a.o_sn = view[3].sn;
  a.lse = return_lse ? lse : nullptr;
  a.slopes = slopes; a.prefix = prefix_lens; a.doc_q = doc_q; a.doc_k = doc_k;
  a.err = reinterpret_cast<int*>(w);
  a.doc_tiles = reinterpret_cast<DocTile*>(w + L.tiles);
  a.part_o = reinterpret_cast<float*>(w + L.part_o);
  a.part_ml = reinterpret_cast<float*>(w + L.part_ml);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (seqlen_k == 0) {
    scored_empty_kernel<<<(unsigned)(((int64_t)batch * heads_q * seqlen_q + 3) / 4), 128, 0, st>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? SAGE_OK : note_cuda_failure(e, "scored attention");
  }
  CUtensorMap maps[3];
  cudaError_t e = cudaSuccess;
  for (int i = 0; i < 3 && e == cudaSuccess; ++i) {
    View& t = view[i];
    int inner = head_dim;
    if (!packed) {
      CopyArgs c{static_cast<const uint16_t*>(t.p), t.sb, t.sh, t.sn, reinterpret_cast<uint16_t*>(w + L.copy[i]),
                 t.heads, t.n, head_dim, L.dp, (int64_t)batch * t.heads * t.n};
      const int64_t blocks = (c.lines + 3) / 4;
      scored_copy_kernel<<<(unsigned)(blocks < 4864 ? blocks : 4864), 128, 0, st>>>(c);
      e = cudaGetLastError();
      t = {c.dst, (int64_t)t.heads * t.n * L.dp, (int64_t)t.n * L.dp, L.dp, t.heads, t.n};
      inner = L.dp;
    }
    // a stride that is never walked (its dimension is 1 long) is given a legal value
    const int64_t sn = t.n > 1 ? t.sn : 128, sh = t.heads > 1 ? t.sh : 128, sb = batch > 1 ? t.sb : 128;
    if (!make_map4(&maps[i], dtype == SAGE_BF16, t.p, inner, t.n, t.heads, batch, sn * 2, sh * 2, sb * 2, 64,
                   i == 0 ? 1 << L.row_bits : 128))
      return note_cuda_failure(cudaErrorInvalidValue, "cuTensorMapEncodeTiled");
  }
  if (e == cudaSuccess && doc_k) {
    scored_setup_kernel<<<dim3(L.k_tiles, batch), 128, 0, st>>>(a);
    e = cudaGetLastError();
  }
  const dim3 grid((unsigned)(heads_kv * L.ctas_kv), (unsigned)blocks_q, (unsigned)(batch * L.splits));
  if (e == cudaSuccess) {
    if (dtype == SAGE_BF16)
      e = L.dp == 64 ? launch_scored<64, true>(a, maps, grid, st) : launch_scored<128, true>(a, maps, grid, st);
    else
      e = L.dp == 64 ? launch_scored<64, false>(a, maps, grid, st) : launch_scored<128, false>(a, maps, grid, st);
  }
  return e == cudaSuccess ? SAGE_OK : note_cuda_failure(e, "scored attention");
}

}  // extern "C"
