// The selective state space scan of a prompt in chunks of 128 tokens on the tensor cores (sm_103a).
//
//   S_t = exp(s_t A) S_{t-1} + s_t x_t B_t^T,   y_t = (S_t C_t + D x_t) silu(z_t)
//
// With L = cumsum(s A) inside a chunk and S_0 the state before it, the recurrence unrolls to
//
//   y_i = e^{L_i} S_0 C_i + sum_{j <= i} M_ij x_j,     M_ij = e^{L_i - L_j} s_j (C_i . B_j)
//   S   = e^{L_last} S_0 + sum_j w_j x_j B_j^T,        w_j  = e^{L_last - L_j} s_j
//
// four matrix products a chunk: the scores C B^T, C S_0^T, M x and (w x)^T B.  Only S links the
// chunks, and only by an elementwise update, so the products of a chunk need nothing but the state.
// A CTA carries the state of 128 rows (one head of dv = 128, or two heads of one key head, 64 rows
// reserved for each) through a run of chunks (a segment: the whole sequence when there are enough
// sequences and heads to fill the device).  All sixteen warps do the elementwise work of each step
// between two block barriers a chunk while one thread issues MMAs that run behind it:
//
//   S (fp32 registers) -> bf16 operand; w x of tokens 0..63    | barrier
//   MMA: C S_0^T, (w x)^T B of tokens 0..63                    | meanwhile M from the scores, the chunk
//                                                              | before's outputs to memory, e^{L_i} (C S_0^T)
//   w x of tokens 64..127                                      | barrier
//   MMA: + M x, (w x)^T B of tokens 64..127, the next scores   | meanwhile outputs, then S
//
// Operands.  x, B and C are used as they come (bf16).  The state and M are rounded to bf16 as operands
// (2^-9 of each term, the size of the outputs' own rounding).  The state itself stays fp32: w x is
// split into three bf16 terms (24 bits together) and each chunk's sum, 128 tokens long, is added to S
// in fp32 outside the tensor core, whose accumulator would truncate.
#pragma once

#include "gdn_ssm.cuh"
#include "gdn_tc.cuh"
#include "gdn_tmap.cuh"

namespace gdn {
namespace ssm {

constexpr int kQ = 128;        // tokens a chunk
constexpr int kThreads = 512;  // 16 warps: warp w reads TMEM lanes 32 (w % 4) .. + 31
constexpr uint32_t kMaxPolls = 1u << 24;
constexpr uint32_t kTmemCols = 512;
// TMEM columns: the scores and, in their place, M in bf16; y; the state's sum; w x in three terms
constexpr uint32_t kColSc = 0, kColY = 128, kColDs = 256, kColXw = 384;

// Segments of a batch: dense sequences have ceil(chunks / len) each; packed ones max(1, ...) each, one
// after the other, `slots` of them at most.
struct Segs {
  const int32_t* cu;     // packed boundaries or null
  const int32_t* order;  // packed, whole sequences: dispatch order (most chunks first) or null
  int B, T;
  int len;     // chunks a segment (0: whole sequences)
  int slots;   // segments of the grid
};

struct Seg {
  int b;            // sequence
  long long bos;    // its first token
  int t0, t1;       // the segment's tokens within it
  int slot;         // index of the segment's stored state
  bool first, last;
};

__device__ __forceinline__ int seg_count(const Segs& g, int len) {
  const int per = g.len * kQ;
  return len <= per ? 1 : (len - 1) / per + 1;
}

// Segment `i` of the grid (every warp finds it for itself); false if there is none.
__device__ __forceinline__ bool find_seg(const Segs& g, int i, Seg& s) {
  int p = 0;  // position in the sequence
  if (g.len == 0) {
    s.b = i;
    if (g.order != nullptr) {
      const int o = g.order[i];
      s.b = o >= 0 && o < g.B ? o : i;
    }
  } else if (g.cu == nullptr) {
    const int n = seg_count(g, g.T);
    s.b = i / n;
    p = i - s.b * n;
  } else {  // the sequence whose segments include i: a running sum over 32 sequences at a time
    const int lane = threadIdx.x & 31;
    int base = 0;
    s.b = -1;
    for (int b0 = 0; b0 < g.B && s.b < 0; b0 += 32) {
      int n = b0 + lane < g.B ? seg_count(g, seq_bounds(g.cu, b0 + lane, g.T).len) : 0, sum = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += y;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, base + sum > i);
      if (hit != 0) {
        const int l = __ffs(hit) - 1;
        s.b = b0 + l;
        p = i - (base + __shfl_sync(0xffffffffu, sum - n, l));
      }
      base += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (s.b < 0) return false;
  }
  const SeqChunk q = seq_bounds(g.cu, s.b, g.T);
  s.bos = q.bos;
  s.slot = i;
  const int per = g.len == 0 ? q.len : g.len * kQ;
  s.t0 = g.len == 0 ? 0 : p * per;
  s.t1 = q.len - s.t0 < per ? q.len : s.t0 + per;
  s.first = p == 0;
  s.last = s.t1 == q.len;
  return true;
}

// PB: state rows reserved for a head (64 or 128; a head of dv = 32 leaves the upper half unused);
// HPC: heads of the CTA.
template <int DK, int PB, int HPC>
struct Cfg {
  static constexpr int kRows = PB * HPC;            // 64 or 128
  static constexpr int kNB = DK > 64 ? 2 : 1;       // 64-wide blocks of B, C and the state
  static constexpr int kXB = kRows / 64;            // 64-wide blocks of x
  static constexpr int kSC = DK / 4;                // state columns a thread holds
  static constexpr int kYC = kRows / 4;             // output columns a thread works on
  // shared memory: two stages of [B][x], one C, the state operand, tables, barriers
  static constexpr int kOffB = 0, kOffX = kNB * 16384, kStage = (kNB + kXB) * 16384;
  static constexpr int kOffC = 2 * kStage;
  static constexpr int kOffS = kOffC + kNB * 16384;
  static constexpr int kOffTab = kOffS + kNB * kRows * 128;
  static constexpr int kTab = HPC * 3 * kQ * 4;     // L, s and w of a chunk
  static constexpr int kOffBar = kOffTab + 2 * kTab;
  static constexpr int kSmemBytes = kOffBar + 256 + 1024;  // + slack for 1024-byte alignment
  static_assert(PB == 64 || (PB == 128 && HPC == 1), "128 rows at most");
  static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void tmem_st8_nowait(uint32_t a, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(a), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st16_nowait(uint32_t a, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(a),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

template <int N>
__device__ __forceinline__ void tmem_load(uint32_t a, float (&v)[N]) {
  static_assert(N == 8 || N == 16 || N == 32, "");
  if constexpr (N == 8) tc::tmem_ld8(a, v);
  else if constexpr (N == 16) tc::tmem_ld16(a, v);
  else tc::tmem_ld32(a, v);
}

// The steps of chunk tokens 4 lane .. + 3 of head h (0 past the chunk's n tokens).
__device__ __forceinline__ void load_steps(const SsmArgs& a, long long t, int n, int h, int lane, float (&d)[4]) {
#pragma unroll
  for (int u = 0; u < 4; ++u) d[u] = 4 * lane + u < n ? ssm_dt(a, t + 4 * lane + u, h) : 0.f;
}

// One warp: the tables of a chunk from its steps.  L in units of log2, inclusive of each token's own
// decay; returns L of the last token in every lane.  The weights' exponents are sums over the tokens after
// each, from the end: as differences of L they would carry the rounding of a strong decay's large L.
// tab: L, s, w (kQ each), or w alone when STATES_ONLY.
template <bool STATES_ONLY>
__device__ __forceinline__ float make_tables(float* tab, const float (&d)[4], float a_log2, int lane) {
  const float e0 = d[0] * a_log2, e1 = d[1] * a_log2, e2 = d[2] * a_log2, e3 = d[3] * a_log2;
  const float own = (e0 + e1) + (e2 + e3);
  float from = own, upto = own;  // sums over the lanes from and up to this one
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float y = __shfl_up_sync(0xffffffffu, upto, o), z = __shfl_down_sync(0xffffffffu, from, o);
    if (lane >= o) upto += y;
    if (lane + o < 32) from += z;
  }
  const float end = __shfl_sync(0xffffffffu, upto, 31);
  float before = __shfl_up_sync(0xffffffffu, upto, 1), after = __shfl_down_sync(0xffffffffu, from, 1);
  if (lane == 0) before = 0.f;
  if (lane == 31) after = 0.f;
  const float4 w = make_float4(exp2f(after + ((e3 + e2) + e1)) * d[0], exp2f(after + (e3 + e2)) * d[1],
                               exp2f(after + e3) * d[2], exp2f(after) * d[3]);
  if (STATES_ONLY) {
    reinterpret_cast<float4*>(tab)[lane] = w;
  } else {
    reinterpret_cast<float4*>(tab)[lane] =
        make_float4(before + e0, before + (e0 + e1), before + ((e0 + e1) + e2), before + own);
    reinterpret_cast<float4*>(tab + kQ)[lane] = make_float4(d[0], d[1], d[2], d[3]);
    reinterpret_cast<float4*>(tab + 2 * kQ)[lane] = w;
  }
  return end;
}

// w x of sixteen tokens t .. t + 15 of state row `row` as three bf16 terms into columns col, col + 32
// and col + 64 (two tokens a column): the A operand of the state's product, 24 bits in all.
__device__ __forceinline__ void split_xw(const unsigned char* xt, const float* w, int row, int t, uint32_t col) {
  uint32_t hi[8], mid[8], lo[8];
  const unsigned char* blk = xt + (row >> 6) * 16384 + (row & 7) * 2;
  const uint32_t ch = (uint32_t)(row & 63) >> 3;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 w4 = *reinterpret_cast<const float4*>(w + t + 4 * i);
    const float wv[4] = {w4.x, w4.y, w4.z, w4.w};
    float v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t raw = *reinterpret_cast<const uint16_t*>(blk + tc::sw128((uint32_t)(t + 4 * i + u), ch));
      v[u] = __uint_as_float(raw << 16) * wv[u];
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int k = 2 * i + u;
      float a = v[2 * u], b = v[2 * u + 1];
      hi[k] = pack_bf16(a, b);
      a -= __uint_as_float(hi[k] << 16);
      b -= __uint_as_float(hi[k] & 0xffff0000u);
      mid[k] = pack_bf16(a, b);
      a -= __uint_as_float(mid[k] << 16);
      b -= __uint_as_float(mid[k] & 0xffff0000u);
      lo[k] = pack_bf16(a, b);
    }
  }
  tmem_st8_nowait(col, hi);
  tmem_st8_nowait(col + 32, mid);
  tmem_st8_nowait(col + 64, lo);
}

// Issue (w x)^T B of 64 tokens (half `hf` of the tile at shared address bt): the small terms first, so
// that the accumulator truncates the large sum's steps only.
template <int DK>
__device__ __forceinline__ void issue_state(uint32_t tmem, uint32_t xw, uint32_t bt, int hf, bool start) {
  constexpr uint32_t kId = tc::idesc_bf16(128, DK, 0, 1);
  const uint64_t bd = tc::sdesc(bt, 16384, 1024, tc::kSw128) + (uint64_t)((hf * 8192) >> 4);
#pragma unroll
  for (int term = 2; term >= 0; --term)
#pragma unroll
    for (int ks = 0; ks < 4; ++ks)
      tc::mma_f16_ta(tmem + kColDs, xw + 32 * term + 8 * ks, bd + (uint64_t)((ks * 2048) >> 4), kId,
                     !(start && term == 2 && ks == 0));
}

}  // namespace ssm
}  // namespace gdn
