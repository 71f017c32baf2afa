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
// sequences and heads to fill the device).  Sixteen worker warps do the elementwise work, one thread
// issues the MMAs and the tile copies, one warp makes the decay tables a chunk ahead; they meet on
// mbarriers only, so that warps drift apart and one's arithmetic covers another's wait.  A chunk's
// outputs are worked on after the next chunk's first operands are out, beside its first products:
//
//   workers: w x of tokens 64..127                                   | MMA: -
//            y = e^{L_i} (C S_0^T); M from the scores; some of silu(z) | MMA: (w x)^T B of 64..127
//            S; the next chunk's S -> bf16 and w x of tokens 0..63     | MMA: y += M x, the next scores
//            the rest of silu(z), outputs                              | MMA: the next (w x)^T B of 0..63 and C S_0^T
//
// What bounds a step (about 8,000 cycles at 128 x 128) is the workers' own path: its instructions (the SM issues in 58%
// of the cycles) and the latency of what they meet: a barrier's state (200 cycles beside running MMAs, hence `peek`),
// TMEM, spilled registers, which come back from L2 (so that little is kept that can be worked out anew, and the gate
// goes through silu only where it is used).  The MMAs take 3,840 cycles of it, the tiles' bytes about 5,600 at the
// device's bandwidth.  32 ragged prompts of 32 heads, 72,102 tokens: 547 to 565 us, 4.4 TB/s of needed bytes.  (Warps
// split into a group that carries the state and one that makes outputs, each with half the warps to hide its latencies:
// 20% slower.  All of the gate through silu beside the state's product, kept in registers until the outputs: 8%.)
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
constexpr int kWorkers = 16;  // worker warp w reads TMEM lanes 32 (w % 4) .. + 31
// A warp that issues and two that make tables (the output pass uses one).  Nineteen warps put five on three of the
// SM's sub-partitions, which caps a thread at 96 registers.
constexpr int kIssueWarp = kWorkers, kTableWarp = kWorkers + 1, kAllocWarp = kWorkers + 2;
constexpr int kThreads = 32 * (kWorkers + 3);
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
  int joined;  // the stored states are start states (else the segments' sums)
  uint32_t polls;  // of a wait, kMaxPolls but in tests (the output pass's whole-warp waits have the constant)
};

struct Seg {
  int b;            // sequence
  int p;            // the segment's place in it
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
  s.p = p;
  s.bos = q.bos;
  s.slot = i;
  const int per = g.len == 0 ? q.len : g.len * kQ;
  s.t0 = g.len == 0 ? 0 : p * per;
  s.t1 = q.len - s.t0 < per ? q.len : s.t0 + per;
  s.first = p == 0;
  s.last = s.t1 == q.len;
  return true;
}

// Tensor maps of a call: boxes of 128 tokens x 64 columns, 128-byte swizzle (out: 32 tokens).
struct Maps {
  CUtensorMap x, b, c, z, out;
};

// PB: state rows reserved for a head (64 or 128; a head of dv = 32 leaves the upper half unused);
// HPC: heads of the CTA.
template <int DK, int PB, int HPC>
struct Cfg {
  static constexpr int kRows = PB * HPC;            // 64 or 128
  static constexpr int kNB = DK > 64 ? 2 : 1;       // 64-wide blocks of B, C and the state
  static constexpr int kXB = kRows / 64;            // 64-wide blocks of x
  static constexpr int kSC = DK / 4;                // state columns a thread holds
  static constexpr int kYC = kRows / 4;             // output columns a thread works on
  // shared memory: two stages of [B][x], one C, the state operand, the gate's tile (in the place of the state
  // operand, once C S^T is done, where there is no room for its own), tables, barriers
  static constexpr int kOffB = 0, kOffX = kNB * 16384, kStage = (kNB + kXB) * 16384;
  static constexpr int kOffC = 2 * kStage;
  static constexpr int kOffS = kOffC + kNB * 16384;
  static constexpr int kSBytes = kNB * kRows * 128 > kXB * 16384 ? kNB * kRows * 128 : kXB * 16384;
  static constexpr int kTabBytes = HPC * 5 * kQ * 4;  // tables of a chunk (the pass of the sums: w of two, decays)
  static constexpr int kBarBytes = 256;               // mbarriers, TMEM base, abort flag, decays, gaps
  static constexpr bool kOwnGate = kOffS + kSBytes + kXB * 16384 + kTabBytes + kBarBytes <= 227 * 1024;
  static constexpr int kOffZ = kOwnGate ? kOffS + kSBytes : kOffS;
  static constexpr int kOffTab = kOwnGate ? kOffZ + kXB * 16384 : kOffS + kSBytes;
  static constexpr int kOffBar = kOffTab + kTabBytes;
  // More than half an SM's, so that two CTAs never share one: each takes all of its TMEM, and one of the output pass
  // that had it would wait for the pass of the sums, which would wait for the TMEM.
  static constexpr int kSmemBytes = kOffBar + kBarBytes > 116 * 1024 ? kOffBar + kBarBytes : 116 * 1024;
  static_assert(PB == 64 || (PB == 128 && HPC == 1), "128 rows at most");
  static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");
};

constexpr uint32_t kMaxPolls = 1u << 18;  // of a wait, 3.7 us each: about a second; then it gives up

// A worker thread's place, worked out anew where it is used: kept from one use to the next it would not fit the
// registers, and with so little of the SM's memory left as L1 a spilled value comes back from L2.
struct Worker {
  int lane, q4, cg, row;  // q4: TMEM lanes 32 q4 .. + 31; cg: its quarter of the columns; row: state row, or token
};
__device__ __forceinline__ Worker worker() {
  int t;
  asm volatile("mov.u32 %0, %%tid.x;" : "=r"(t));
  return {t & 31, (t >> 5) & 3, t >> 7, t & 127};
}

// Whether a phase has ended, asked some time before it matters: the answer takes about 200 cycles.
__device__ __forceinline__ uint32_t peek(uint64_t* bar, uint32_t par) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(done)
      : "r"(smem_u32(bar)), "r"(par));
  return done;
}

// A box of a tile from shared memory to global memory, in the thread's next bulk group.
__device__ __forceinline__ void tma_store_2d(const void* map, uint32_t src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];\n" ::"l"(map), "r"(x),
               "r"(y), "r"(src)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;\n" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;\n" ::: "memory"); }

__device__ __forceinline__ void tma_prefetch_l2_2d(const void* map, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];\n" ::"l"(map), "r"(x), "r"(y)
               : "memory");
}

__device__ __forceinline__ void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(smem_u32(bar)) : "memory");
}

// Sixteen lanes (from taddr's) of eight columns: register 2 j + i of thread l holds lane l / 4 + 8 i,
// column 4 j + l % 4 -- the layout of transposed ldmatrix fragments.
__device__ __forceinline__ void tmem_st_16x128b_x2(uint32_t a, const uint32_t (&v)[4]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1,%2,%3,%4};\n" ::"r"(a), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3])
               : "memory");
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

// dt of chunk tokens 4 lane .. + 3 of head h, loaded a chunk ahead (the last token's past the chunk's n), and
// the steps it stands for (0 past n).
__device__ __forceinline__ void load_dt(const SsmArgs& a, long long t, int n, int h, int lane, uint32_t (&d)[4]) {
#pragma unroll
  for (int u = 0; u < 4; ++u) d[u] = ssm_load_dt(a, t + min(4 * lane + u, n - 1), h);
}
__device__ __forceinline__ void to_steps(const SsmArgs& a, int n, float bias, int lane, const uint32_t (&r)[4],
                                         float (&d)[4]) {
#pragma unroll
  for (int u = 0; u < 4; ++u) d[u] = 4 * lane + u < n ? ssm_step_of(a, r[u], bias) : 0.f;
}

// One warp: the tables of a chunk from its steps, tokens 4 lane .. + 3 in each lane, in units of log2.  No exponent is
// the difference of two sums over more than 32 tokens, since it would carry the rounding of what it does not contain
// (a strong decay's large L, before a pair of tokens whose own decay is weak).  With the chunk in blocks of 32 tokens,
// M's exponent L_i - L_j + log2 s_j is
//   L - K          in one block, L inclusive of a token's own decay and from its block's start, K = L - log2 |s|;
//   L + gap - far  between blocks, the gap the sum over the blocks between, far = -(the sum after j in its block)
//                  - log2 |s_j|.
// A step below zero (there are none with softplus) leaves its sign to M and has it in w, a zero w too.
// The weights' exponents are sums over the tokens after each, from the chunk's end.  A token's decay below 2^-160 is 0
// in fp32 and counts as 2^-160, which keeps L above -5,120: its roundings (2^-12) stay below that of M to bf16 (2^-9).
struct Tables {
  float4 L, K, far, w, e;  // e: 2^(the sum up to a token)
  float2 gap;              // between the lane's block and blocks 0 and 1
  float end;               // the sum over the chunk, in every lane
};
__device__ __forceinline__ Tables make_tables(const float (&d)[4], float a_log2, int lane) {
  constexpr float kLeast = -160.f;
  const float e0 = max_nan(d[0] * a_log2, kLeast), e1 = max_nan(d[1] * a_log2, kLeast);
  const float e2 = max_nan(d[2] * a_log2, kLeast), e3 = max_nan(d[3] * a_log2, kLeast);
  const float own = (e0 + e1) + (e2 + e3);
  const int at = lane & 7, block = lane >> 3;
  float from = own, upto = own;  // sums over the block's lanes from and up to this one
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    const float y = __shfl_up_sync(0xffffffffu, upto, o, 8), z = __shfl_down_sync(0xffffffffu, from, o, 8);
    if (at >= o) upto += y;
    if (at + o < 8) from += z;
  }
  const float b0 = __shfl_sync(0xffffffffu, upto, 7), b1 = __shfl_sync(0xffffffffu, upto, 15);
  const float b2 = __shfl_sync(0xffffffffu, upto, 23), b3 = __shfl_sync(0xffffffffu, upto, 31);
  float before = __shfl_up_sync(0xffffffffu, upto, 1, 8), after = __shfl_down_sync(0xffffffffu, from, 1, 8);
  if (at == 0) before = 0.f;
  if (at == 7) after = 0.f;
  Tables t;
  t.end = (b0 + b1) + (b2 + b3);
  t.gap = make_float2(block == 3 ? b1 + b2 : b1, b2);
  const float earlier = block == 0 ? 0.f : block == 1 ? b0 : block == 2 ? b0 + b1 : (b0 + b1) + b2;
  const float later = block == 0 ? b1 + (b2 + b3) : block == 1 ? b2 + b3 : block == 2 ? b3 : 0.f;
  const float4 rest = make_float4(after + ((e3 + e2) + e1), after + (e3 + e2), after + e3, after);
  const float4 size = make_float4(log2f(fabsf(d[0])), log2f(fabsf(d[1])), log2f(fabsf(d[2])), log2f(fabsf(d[3])));
  t.w = make_float4(exp2f(later + rest.x) * d[0], exp2f(later + rest.y) * d[1], exp2f(later + rest.z) * d[2],
                    exp2f(later + rest.w) * d[3]);
  t.L = make_float4(before + e0, before + (e0 + e1), before + ((e0 + e1) + e2), before + own);
  t.e = make_float4(exp2f(earlier + t.L.x), exp2f(earlier + t.L.y), exp2f(earlier + t.L.z), exp2f(earlier + t.L.w));
  t.K = make_float4(t.L.x - size.x, t.L.y - size.y, t.L.z - size.z, t.L.w - size.w);
  t.far = make_float4(-rest.x - size.x, -rest.y - size.y, -rest.z - size.z, -rest.w - size.w);
  return t;
}

// Sixteen bf16, their signs turned where those of w (in shared memory) are set.
__device__ __forceinline__ void turn_signs(uint32_t (&m)[8], const float* w) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint2 s = *reinterpret_cast<const uint2*>(w + 2 * j);
    m[j] ^= ((s.x & 0x80000000u) >> 16) | (s.y & 0x80000000u);
  }
}

// x of sixteen tokens t .. t + 15 and state rows row0 .. + 31 as a warp multiplies it by w (in shared memory beside
// running MMAs both take hundreds of cycles, so they are loaded some time before they are split).
struct XwTiles {
  uint32_t x[2][4];
  float2 w[2];
};
__device__ __forceinline__ void load_xw(XwTiles& v, const unsigned char* xt, const float* w, int lane, int row0,
                                        int t) {
  const uint32_t tok = (uint32_t)(t + ((lane >> 4) << 3) + (lane & 7));  // this lane's row of the four 8 x 8 tiles
#pragma unroll
  for (int rh = 0; rh < 2; ++rh) {
    const int r = row0 + 16 * rh + (lane & 8);
    ldsm_x4_t(v.x[rh], xt + (r >> 6) * 16384 + tc::sw128(tok, (uint32_t)(r & 63) >> 3));
  }
  v.w[0] = *reinterpret_cast<const float2*>(w + t + 2 * (lane & 3));
  v.w[1] = *reinterpret_cast<const float2*>(w + t + 8 + 2 * (lane & 3));
}

// w x as three bf16 terms into columns col, col + 32 and col + 64 (two tokens a column) of the warp's lanes: the A
// operand of the state's product.  The terms take fp32's 24 bits eight at a time, so nothing is lost.
__device__ __forceinline__ void split_xw(const XwTiles& tiles, uint32_t col) {
#pragma unroll
  for (int rh = 0; rh < 2; ++rh) {
    const uint32_t(&x)[4] = tiles.x[rh];
    uint32_t hi[4], mid[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // tiles (tokens 0..7, 8..15) x (rows 0..7, 8..15), rows innermost
      const float2 v =
          mul2(make_float2(__uint_as_float(x[i] << 16), __uint_as_float(x[i] & 0xffff0000u)), tiles.w[i >> 1]);
      const uint32_t a = __float_as_uint(v.x), b = __float_as_uint(v.y);
      hi[i] = __byte_perm(a, b, 0x7632);
      const float2 m = fma2(make_float2(__uint_as_float(a & 0xffff0000u), __uint_as_float(b & 0xffff0000u)),
                            make_float2(-1.f, -1.f), v);
      const uint32_t c = __float_as_uint(m.x), d = __float_as_uint(m.y);
      mid[i] = __byte_perm(c, d, 0x7632);
      const float2 l = fma2(make_float2(__uint_as_float(c & 0xffff0000u), __uint_as_float(d & 0xffff0000u)),
                            make_float2(-1.f, -1.f), m);
      lo[i] = __byte_perm(__float_as_uint(l.x), __float_as_uint(l.y), 0x7632);
    }
    const uint32_t at = col + ((uint32_t)(16 * rh) << 16);
    tmem_st_16x128b_x2(at, hi);
    tmem_st_16x128b_x2(at + 32, mid);
    tmem_st_16x128b_x2(at + 64, lo);
  }
}

// Issue (w x)^T B of 64 tokens (half `hf` of the tile at shared address bt) into columns `sum`: the small
// terms first, so that the accumulator truncates the large sum's steps only.
template <int DK>
__device__ __forceinline__ void issue_state(uint32_t sum, uint32_t xw, uint32_t bt, int hf, bool start) {
  constexpr uint32_t kId = tc::idesc_bf16(128, DK, 0, 1);
  const uint64_t bd = tc::sdesc(bt, 16384, 1024, tc::kSw128) + (uint64_t)((hf * 8192) >> 4);
#pragma unroll
  for (int term = 2; term >= 0; --term)
#pragma unroll
    for (int ks = 0; ks < 4; ++ks)
      tc::mma_f16_ta(sum, xw + 32 * term + 8 * ks, bd + (uint64_t)((ks * 2048) >> 4), kId,
                     !(start && term == 2 && ks == 0));
}

}  // namespace ssm
}  // namespace gdn
