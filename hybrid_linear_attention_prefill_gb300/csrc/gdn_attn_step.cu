// Attention of one token of every sequence over a paged cache (sm_103a; gdn_attn.cuh has the mathematics).
//
// Every visible key and value is read once for two products with a handful of queries: bandwidth bounds it.
//
//   scores   S^T [16 keys x 8 heads] = K Q^T      `mma.sync` products; asynchronous copies bring 16 keys and values a
//   outputs  O^T [16 columns x 8 heads] += V^T P  time into a warp's ring in shared memory, and ldmatrix takes the
//                                                 operands from there (transposed for V); the weights, keys by heads as
//                                                 the scores come, are transposed by `movmatrix`
//
// The ring keeps 128 KB of an SM on their way whatever the products do, and a warp meets no other until its sequence
// ends; a block's place in the cache is looked up by a lane for 32 blocks at a time.  (Loads straight into registers
// kept as many bytes on their way with bf16, half as many with e4m3, whose products also took twice the instructions:
// 160 us for 32 long requests over an 8-bit cache where the ring took 111.)  With an 8-bit cache two blocks are taken
// together, since the chain of one block's steps, not the bytes, bound it (136 us where two took 111).
//
// Work.  A unit is 64 keys, 16 for each warp of a CTA.  The units of all sequences and key heads, one after the
// other, are dealt out in equal runs to as many CTAs as are resident, whatever the lengths; a warp keeps its own
// maxima, sums and outputs, and the CTA joins its warps' where a sequence (or the run) ends, while the next one's first
// blocks are on their way.  A sequence that is cut leaves partial sums in the workspace; the CTA that finishes its last
// part joins them in the runs' order, so results do not depend on which that is.  Where there are few sequences and key
// heads, a run stays within one: a second item, with its own queries, lookups and join, costs it 5 us (one request of 3,001
// tokens 17.3 us, 13.0 since; of 4,096, whose units divide, 12.2 and 12.5, on the device).  More than 16 heads of a key
// head are taken 16 at a time.
//
// Over a bf16 cache a weight is two bf16 operands, its upper 16 bits and what they leave: 2^-16 of it is lost, not the 2^-9
// of one operand, and the tensor cores, which wait for bytes, take the second product in their stride.
//
// A running maximum stays in use until a score is 2^8 above it (as for prompts), so that a step needs a vote and no
// exchange.  With an 8-bit cache the products are of fp16: every e4m3 value is one; the queries are scaled by a power
// of two a head to fit; weights are rounded to 11 bits, next to the values' 4.  fp16 loses bits below 2^-14, so the weights are
// held relative to 2^-7 of the maximum: up to 2^15 then, and each is off by 2^-25, 2^-32 of their sum, at most.
//
// Measured on one GB300, L2 cold, call after call: 128 ragged requests (1.16 GB of keys and values) 182 us, 6.4 TB/s; 32
// long requests over an 8-bit cache (531 MB) 91.5 us, 5.8 TB/s; a window of 1,024 for 128 requests (541 MB) 90.8 us; one
// request of 4,096 tokens 12.3 us (32 parts a head).  A call costs about 12 us beside its bytes: launch, three dependent
// first reads (lengths, table, keys), the last join.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <type_traits>

#include "gdn_attn.cuh"
#include "gdn_internal.h"

namespace gdn {

namespace {

using attn::Seen;
using attn::StepArgs;

constexpr int kWarps = 4, kThreads = 32 * kWarps, kCtas = 2;  // (a CTA, an SM)
constexpr int kBlock = 16;                  // keys a warp takes at a time
constexpr int kMaxHeads = 16;               // of a key head at a time
constexpr float kLazy = 8.f;
// Runs lie apart where there are this many CTAs for a sequence's key head (304 CTAs; 5 requests of 8 heads 15.6 us instead
// of 18.7, 8 requests 19.8 instead of 21.0; 18 requests, where two suffice, 40.9 instead of 40.5).
constexpr int kFew = 4;
constexpr int kBadPage = 64;                // GDN_STATUS_BAD_PAGE

// Partial sums of a run's two ends: [2 runs][heads][d], then maxima and sums [2 runs][heads].
struct Work {
  float* sums;
  float2* stats;
  int* counters;  // parts of a (sequence, key head) that are done; zero between calls
};

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// 16 or 8 bytes into shared memory, zeros where not `there`.
__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(to), "l"(from), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t to, const void* from, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;\n" ::"r"(to), "l"(from), "r"(there ? 8 : 0) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;\n" ::"n"(kLeft) : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t at, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t at, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
// Four e4m3 values as fp16.
__device__ __forceinline__ void widen_e4m3(uint32_t x, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(x));
}

// What is left of a weight without its lower 16 bits.  A weight above 0 leaves something above 0, so that an infinity among
// the values stays one.
__device__ __forceinline__ float cut_off(float w) {
  return fmaxf(w - __uint_as_float(__float_as_uint(w) & 0xffff0000u), fminf(w, 0x1p-126f));
}

// A warp's ring: kRing times kPer blocks of 16 keys and their values.  A row is padded or its 16-byte pieces are permuted, so that
// eight rows' pieces of a column lie in different banks.
template <int NT, int NC, bool E4M3>
struct Ring {
  static constexpr int kSize = E4M3 ? 1 : 2, kBytes = 32 * NC * kSize;  // of a value, of a row
  static constexpr bool kXor = kBytes % 128 == 0;
  static constexpr int kPitch = kXor ? kBytes : kBytes + 16, kTile = kBlock * kPitch, kPieces = kBytes / 16;
  static constexpr int kPer = E4M3 ? 2 : 1, kRing = 3, kSlot = kPer * 2 * kTile;
  static constexpr int kRow = 32 * NC + 4;  // a head's sums, padded
  static constexpr int kOffSums = kWarps * kRing * kSlot, kOffStat = kOffSums + kWarps * 8 * kRow * 4;
  static constexpr int kSmem = kOffStat + kWarps * 8 * 8 + 16;
  static_assert(kSmem <= 113 * 1024, "two CTAs an SM");
  __device__ static __forceinline__ int at(int row, int piece) {
    return row * kPitch + 16 * (kXor ? piece ^ (row & 7) : piece);
  }
};

__device__ __forceinline__ long long inclusive(long long x, int lane) {  // the sum up to this lane
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}
// Of numbers that are not negative: in 32 bits where they fit, which is many times as fast.
__device__ __noinline__ long long long_quotient(long long x, long long y) { return x / y; }
__device__ __forceinline__ long long quotient(long long x, long long y) {
  return ((x | y) >> 32) == 0 ? (long long)((uint32_t)x / (uint32_t)y) : long_quotient(x, y);
}

// What a part's sums (maximum, sum of weights) are multiplied by to be relative to `top`: nothing of a part that has
// seen nothing (or NaN, where its sum is that).
__device__ __forceinline__ float share(const float2& part, float top) {
  return part.x == -INFINITY ? part.y : ex2_approx(part.x - top);
}
__device__ __forceinline__ float4 add(const float4& x, float f, const float4& y) {
  return make_float4(fmaf(f, y.x, x.x), fmaf(f, y.y, x.y), fmaf(f, y.z, x.z), fmaf(f, y.w, x.w));
}

// A sequence's blocks of 16 keys with something to see: [0, s) and [a, z); the last is count - 1.
struct Blocks {
  int n, s, a, count;
  Seen seen;
};
__device__ __forceinline__ Blocks blocks_of(const StepArgs& a, int b) {
  Blocks r;
  const long long most = (long long)a.W * a.page;
  const int n = a.lens[b];
  r.n = n < 0 ? 0 : n < most ? n : (int)most;
  r.seen = attn::seen_by(a.view, r.n - 1);
  r.a = r.seen.lo / kBlock;
  r.s = min((r.seen.sink_end + kBlock - 1) / kBlock, r.a);
  r.count = r.s + (r.n + kBlock - 1) / kBlock - r.a;
  return r;
}
// (one at least, so that every row is written)
__device__ __forceinline__ int units_of(int blocks) { return blocks > kWarps ? (blocks + kWarps - 1) / kWarps : 1; }

}  // namespace

// NT: heads in eights; NC: columns in 32s; groups: parts of a key head's heads.
template <int NT, int NC, bool E4M3>
__global__ void __launch_bounds__(kThreads, kCtas)
gdn_attn_step_kernel(const StepArgs a, int groups, int heads, float scale_log2, int wide, Work work,
                     int* __restrict__ err) {
  using R = Ring<NT, NC, E4M3>;
  constexpr float kUp = E4M3 ? 7.f : 0.f;  // log2 of the maximum's weight
  extern __shared__ __align__(128) unsigned char sm[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int G = a.Hq / a.Hkv, per_seq = a.Hkv * groups;
  float(*so)[8][R::kRow] = reinterpret_cast<float(*)[8][R::kRow]>(sm + R::kOffSums);
  float2(*stat)[8] = reinterpret_cast<float2(*)[8]>(sm + R::kOffStat);  // maximum (log2) and sum
  int* last = reinterpret_cast<int*>(sm + R::kOffStat + kWarps * 8 * 8);
  const uint32_t ring = smem_u32(sm) + warp * R::kRing * R::kSlot;

  // This CTA's run of units, and the sequence that it begins in: every lane counts a share of the sequences, then the
  // lanes look at the share where the run begins.  With `apart` a run stays within a sequence's key head.
  const int share_of = (a.B + 31) / 32;
  long long mine = 0;
#pragma unroll 4
  for (int i = 0; i < share_of; ++i) {
    const int x = lane * share_of + i;
    mine += x < a.B ? units_of(blocks_of(a, x).count) : 0;
  }
  const int units_here = (int)mine;
  mine *= per_seq;
  long long upto = inclusive(mine, lane), total = __shfl_sync(0xffffffffu, upto, 31);
  long long per_run = quotient(total + gridDim.x - 1, gridDim.x);
  const bool apart = share_of == 1 && a.B * per_seq <= (int)gridDim.x / kFew;
  if (apart) {  // the shortest runs, in steps of a sixteenth, of which there are few enough; from here on, runs are counted
    const int units = units_here;
    int per = (int)per_run, runs;
#pragma unroll 1
    for (;; per += (per + 15) / 16) {
      runs = (units + per - 1) / per * per_seq;
      if (__reduce_add_sync(0xffffffffu, runs) <= (int)gridDim.x) break;
    }
    per_run = per;
    mine = runs;
    upto = inclusive(mine, lane);
    total = __shfl_sync(0xffffffffu, upto, 31);
  }
  long long u0 = apart ? blockIdx.x : blockIdx.x * per_run;
  if (u0 >= total) return;
  const long long u1 = apart ? u0 + 1 : min(u0 + per_run, total);
  const int l0 = __ffs(__ballot_sync(0xffffffffu, upto > u0)) - 1;
  int b = l0 * share_of;
  long long before = __shfl_sync(0xffffffffu, upto - mine, l0);  // of the sequences before b
#pragma unroll 1
  for (int i = 0; share_of > 1; i += 32) {  // (the share has it: a sequence behind the share's last is not reached)
    const int x = b + lane;
    const long long u =
        i + lane < share_of && x < a.B ? (long long)units_of(blocks_of(a, x).count) * per_seq : 0;
    const long long sum = before + inclusive(u, lane);
    const unsigned hit = __ballot_sync(0xffffffffu, sum > u0);
    const int l = hit != 0 ? __ffs(hit) - 1 : 31;
    before = __shfl_sync(0xffffffffu, hit != 0 ? sum - u : sum, l);
    b += hit != 0 ? l : 32;
    if (hit != 0 || i + 32 >= share_of) break;
  }
  Blocks blk = blocks_of(a, b);
  int units = units_of(blk.count);
  const int parts = apart ? (units + (int)per_run - 1) / (int)per_run : units;  // of an item
  int item = (int)quotient(u0 - before, parts), first = (int)((u0 - before) - (long long)item * parts);
  const int part_of = first;
  if (apart) first *= (int)per_run;
  int todo = 0, hk = 0, h0 = 0, nh = 0;

  // ---- the item's keys and values on their way: the pages of 32 of this warp's blocks at a time, a lane each
  int page = -1, in_page = 0, page_after = -1, in_page_after = 0;
  // the first key of this warp's i-th block, -1 behind the last
  auto key_of = [&](int i) {
    const int n = (first + i) * kWarps + warp;
    return i < todo && n < blk.count ? kBlock * (n < blk.s ? n : blk.a + n - blk.s) : -1;
  };
  auto look_up = [&](int i) {
    const int key = key_of(i + lane);
    page_after = -1;
    if (key >= 0) {
      const int x = key / a.page;
      in_page_after = key - x * a.page;
      page_after = a.table[b * a.table_stride + x];
      if (page_after < 0 || page_after >= a.blocks) {
        page_after = -1;
        atomicOr(err, kBadPage);
      }
    }
  };
  auto sees = [&](int key) { return key < blk.n && (key >= blk.seen.lo || key < blk.seen.sink_end); };
  auto sees_all = [&](int key) {
    return key + kBlock <= blk.n && (key >= blk.seen.lo || key + kBlock <= blk.seen.sink_end);
  };
  int slot = 0, put_slot = 0;  // of the ring: where the next block is, where one goes
  uint32_t filled = 0;         // which of the ring's blocks are there
  auto fetch = [&](int i) {
    if ((i * R::kPer & 31) == 0) {
      page = page_after;
      in_page = in_page_after;
      look_up(i * R::kPer + 32);
    }
    int pg[R::kPer], at[R::kPer];
    uint32_t any = 0;
#pragma unroll
    for (int x = 0; x < R::kPer; ++x) {
      pg[x] = __shfl_sync(0xffffffffu, page, (i * R::kPer + x) & 31);
      at[x] = __shfl_sync(0xffffffffu, in_page, (i * R::kPer + x) & 31);
      any |= (uint32_t)(pg[x] >= 0) << x;
    }
    if (any != 0) {
#pragma unroll
      for (int x = 0; x < R::kPer; ++x) {
        const int key = key_of(i * R::kPer + x);
        const bool all = pg[x] >= 0 && sees_all(key);
        const long long from = ((long long)hk * a.page + at[x]) * a.d;
        const unsigned char* kp = static_cast<const unsigned char*>(a.kc) + ((long long)max(pg[x], 0) * a.kbs + from) * R::kSize;
        const unsigned char* vp = static_cast<const unsigned char*>(a.vc) + ((long long)max(pg[x], 0) * a.vbs + from) * R::kSize;
        const uint32_t to = ring + put_slot * R::kSlot + x * 2 * R::kTile;
        // (a value that is not seen is not read: zero times it might not be zero)
        if (!E4M3 || wide) {
#pragma unroll
          for (int e = 0; e < kBlock * R::kPieces; e += 32) {
            const int row = (e + lane) / R::kPieces, piece = (e + lane) - row * R::kPieces;
            const bool there = 16 * piece < a.d * R::kSize && (all || (pg[x] >= 0 && sees(key + row)));
            const int y = there ? row * a.d * R::kSize + 16 * piece : 0;
            copy16(to + R::at(row, piece), kp + y, there);
            copy16(to + R::kTile + R::at(row, piece), vp + y, there);
          }
        } else {
#pragma unroll 1
          for (int e = 0; e < kBlock * R::kPieces * 2; e += 32) {
            const int row = (e + lane) / (2 * R::kPieces), piece = (e + lane) - row * 2 * R::kPieces;
            const bool there = 8 * piece < a.d && (all || (pg[x] >= 0 && sees(key + row)));
            const int y = there ? row * a.d + 8 * piece : 0, z = R::at(row, piece >> 1) + 8 * (piece & 1);
            copy8(to + z, kp + y, there);
            copy8(to + R::kTile + z, vp + y, there);
          }
        }
      }
    }
    copies_end();
    filled = (filled & ~(((1u << R::kPer) - 1u) << R::kPer * put_slot)) | any << R::kPer * put_slot;
    if (++put_slot == R::kRing) put_slot = 0;
  };
  uint32_t q[NT][2 * NC][2];  // queries: head g of each eight, the columns that a product's operand has
  auto begin = [&]() {
    todo = (int)min((long long)(units - first), apart ? per_run : u1 - u0);
    hk = item / groups;
    h0 = hk * G + (item - hk * groups) * heads;
    nh = min(heads, (hk + 1) * G - h0);  // heads of this item
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const __nv_bfloat16* row = a.q + b * a.qs + (long long)(h0 + 8 * t + g) * a.d;
#pragma unroll
      for (int i = 0; i < 2 * NC; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int col = 16 * i + (E4M3 ? 4 * c + 2 * k : 2 * c + 8 * k);
          q[t][i][k] = 8 * t + g < nh && col < a.d ? *reinterpret_cast<const uint32_t*>(row + col) : 0u;
        }
    }
    look_up(0);
    put_slot = slot;
#pragma unroll 1
    for (int i = 0; i < R::kRing - 1; ++i) fetch(i);
  };
  begin();

  while (true) {
    float scale[NT][2];  // of heads 2 c and 2 c + 1
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      scale[t][0] = scale[t][1] = scale_log2;
      if constexpr (E4M3) {
        // to below 2 by a power of two, which the scale takes back
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < 2 * NC; ++i)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float2 f = widen2(q[t][i][k]);
            top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
          }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        int e = (int)(__float_as_uint(top) >> 23) - 127;
        e = e > 127 ? 0 : min(max(e, -100), 126);  // (infinities stay)
        const float down = __uint_as_float((uint32_t)(127 - e) << 23), up = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
        for (int i = 0; i < 2 * NC; ++i)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float2 f = widen2(q[t][i][k]);
            q[t][i][k] = pack_f16(f.x * down, f.y * down);
          }
        const float ks = a.kscale[hk];
        scale[t][0] *= ks * __shfl_sync(0xffffffffu, up, 8 * c);  // lane 4 h has head h's
        scale[t][1] *= ks * __shfl_sync(0xffffffffu, up, 8 * c + 4);
      }
    }

    float o[NT][2 * NC][4] = {};
    float m[NT][2], l[NT][2];  // what weights are relative to (log2), their sum
#pragma unroll
    for (int t = 0; t < NT; ++t) m[t][0] = m[t][1] = -INFINITY, l[t][0] = l[t][1] = 0.f;

#pragma unroll 1
    for (int i = 0; i * R::kPer < todo; ++i) {
      const uint32_t there = filled >> R::kPer * slot & ((1u << R::kPer) - 1u);
      copies_wait<R::kRing - 2>();
      __syncwarp();  // every lane's copies of these blocks are there, and the blocks before are read
      fetch(i + R::kRing - 1);
      __syncwarp();
      if (there != 0) {
        const uint32_t at = ring + slot * R::kSlot;
        float s[R::kPer][NT][4] = {};
#pragma unroll
        for (int j = 0; j < (E4M3 ? NC : 2 * NC); ++j)
#pragma unroll
          for (int x = 0; x < R::kPer; ++x) {
            uint32_t r[4];
            ldmatrix4(at + x * 2 * R::kTile + R::at(lane & 15, 2 * j + (lane >> 4)), r);
            if constexpr (E4M3) {
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                uint32_t ka[4];
                widen_e4m3(r[2 * y], ka[0], ka[2]);
                widen_e4m3(r[2 * y + 1], ka[1], ka[3]);
#pragma unroll
                for (int t = 0; t < NT; ++t) mma_f16(s[x][t], ka, q[t][2 * j + y][0], q[t][2 * j + y][1]);
              }
            } else {
#pragma unroll
              for (int t = 0; t < NT; ++t) mma_bf16(s[x][t], r, q[t][j][0], q[t][j][1]);
            }
          }
        bool above = false;
#pragma unroll
        for (int x = 0; x < R::kPer; ++x) {
          const int key = key_of(i * R::kPer + x);
          const bool some = there >> x & 1u, all = some && sees_all(key);
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              s[x][t][k] *= scale[t][k & 1];
              if (!all && (!some || !sees(key + g + 8 * (k >> 1)))) s[x][t][k] = -INFINITY;
              above |= s[x][t][k] > m[t][k & 1] + (kUp + kLazy);
            }
        }
        if (__any_sync(0xffffffffu, above)) {
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float top = fmaxf(s[0][t][k], s[0][t][k + 2]);
#pragma unroll
              for (int x = 1; x < R::kPer; ++x) top = fmaxf(top, fmaxf(s[x][t][k], s[x][t][k + 2]));
#pragma unroll
              for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
              top -= kUp;
              if (top > m[t][k]) {
                const float f = ex2_approx(m[t][k] - top);  // (0 at first)
                m[t][k] = top;
                l[t][k] *= f;
#pragma unroll
                for (int x = 0; x < 2 * NC; ++x) o[t][x][k] *= f, o[t][x][k + 2] *= f;
              }
            }
        }
        uint32_t p[R::kPer][NT][2], rest[R::kPer][NT][2];  // weights, and with bf16 what their rounding leaves
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const float base[2] = {m[t][0] == -INFINITY ? 0.f : m[t][0], m[t][1] == -INFINITY ? 0.f : m[t][1]};
#pragma unroll
          for (int x = 0; x < R::kPer; ++x) {
            float w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              w[k] = ex2_approx(s[x][t][k] - base[k & 1]);
              l[t][k & 1] += w[k];
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              if constexpr (E4M3) {
                p[x][t][k] = transposed(pack_f16(w[2 * k], w[2 * k + 1]));
              } else {
                p[x][t][k] = transposed(__byte_perm(__float_as_uint(w[2 * k]), __float_as_uint(w[2 * k + 1]), 0x7632));
                rest[x][t][k] = transposed(pack_bf16(cut_off(w[2 * k]), cut_off(w[2 * k + 1])));
              }
            }
          }
        }
        const int v_row = (lane & 7) + (lane >> 4) * 8, v_piece = lane >> 3 & 1;
#pragma unroll
        for (int x = 0; x < R::kPer; ++x)
#pragma unroll
          for (int j = 0; j < (E4M3 ? NC : 2 * NC); ++j) {
            uint32_t r[4];
            ldmatrix4_trans(at + (x * 2 + 1) * R::kTile + R::at(v_row, 2 * j + v_piece), r);
            if constexpr (E4M3) {
              // a lane's four bytes: two keys' two columns; keys 8 on are in the last two
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                uint32_t va[4];
                widen_e4m3(__byte_perm(r[y], 0, 0x3120), va[0], va[1]);
                widen_e4m3(__byte_perm(r[y + 2], 0, 0x3120), va[2], va[3]);
#pragma unroll
                for (int t = 0; t < NT; ++t) mma_f16(o[t][2 * j + y], va, p[x][t][0], p[x][t][1]);
              }
            } else {
#pragma unroll
              for (int t = 0; t < NT; ++t) {
                mma_bf16(o[t][j], r, p[x][t][0], p[x][t][1]);
                mma_bf16(o[t][j], r, rest[x][t][0], rest[x][t][1]);
              }
            }
          }
      }
      if (++slot == R::kRing) slot = 0;
    }

    // the next item's blocks are on their way while this one's sums are joined
    const int at_b = b, at_item = item, at_hk = hk, at_h0 = h0, at_nh = nh, parts_units = units;
    const bool from_start = first == 0, whole = from_start && todo == units;
    const long long at_start = before + (long long)item * units;
    u0 += apart ? 1 : todo;
    const bool more = u0 < u1;
    if (more) {
      first = 0;
      if (++item == per_seq) {
        item = 0;
        before += (long long)units * per_seq;
        blk = blocks_of(a, ++b);
        units = units_of(blk.count);
      }
      __syncwarp();
      begin();
    }

    const int index = 2 * blockIdx.x + (from_start ? 1 : 0);
    const float vs = E4M3 ? a.vscale[at_hk] : 1.f;
    // a head's quotient to its row (four columns), and the log of its sum
    auto put = [&](int h, int col, const float4& x, float top, float sum) {
      const long long row = (long long)at_b * a.Hq + at_h0 + h;
      const float inv = sum == 0.f ? 0.f : vs / sum;
      const float2 f[2] = {{x.x * inv, x.y * inv}, {x.z * inv, x.w * inv}};
      *reinterpret_cast<uint2*>(a.out + row * a.d + col) = sum == 0.f ? make_uint2(0, 0) : narrow4(f);
      if (a.lse != nullptr && col == 0) a.lse[row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * attn::kLn2;
    };
    const int quads = a.d / 4;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      __syncthreads();  // what was there before is read
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float sum = l[t][k];
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
        const int h = 2 * c + k;
        if (g == 0) stat[warp][h] = make_float2(m[t][k], sum);
#pragma unroll
        for (int x = 0; x < 2 * NC; ++x) {
          so[warp][h][16 * x + (E4M3 ? 2 * g : g)] = o[t][x][k];
          so[warp][h][16 * x + (E4M3 ? 2 * g + 1 : g + 8)] = o[t][x][k + 2];
        }
      }
      __syncthreads();
#pragma unroll 1
      for (int x = tid; x < min(at_nh - 8 * t, 8) * quads; x += kThreads) {
        const int h = x / quads, col = 4 * (x - h * quads);
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, stat[w][h].x);
        float4 all4 = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float2 st = stat[w][h];
          const float f = share(st, top);
          const float4 y = *reinterpret_cast<const float4*>(&so[w][h][col]);
          sum = fmaf(f, st.y, sum);
          all4 = add(all4, f, y);
        }
        if (whole) {
          put(8 * t + h, col, all4, top, sum);
        } else {
          const long long to = index * kMaxHeads + 8 * t + h;
          *reinterpret_cast<float4*>(work.sums + to * attn::kMaxDim + col) = all4;
          if (col == 0) work.stats[to] = make_float2(top, sum);
        }
      }
    }
    if (!whole) {
      // the run that finishes the last part joins them all
      auto run_of = [&](long long u) { return (int)quotient(u, per_run); };
      const int r0 = apart ? (int)blockIdx.x - part_of : run_of(at_start);
      const int r1 = apart ? r0 + parts - 1 : run_of(at_start + parts_units - 1);
      int* counter = work.counters + (long long)at_b * per_seq + at_item;
      __threadfence();
      __syncthreads();
      if (tid == 0) *last = atomicAdd(counter, 1) == r1 - r0;
      __syncthreads();
      if (*last) {
        __threadfence();
        if (tid == 0) *counter = 0;
        // their maxima and sums into shared memory, as many parts at a time as fit; a thread has four columns of a head
        float2* const part = reinterpret_cast<float2*>(so);
        const int fit = kWarps * 8 * R::kRow / 2 / at_nh;
#pragma unroll 1
        for (int x0 = 0; x0 < at_nh * quads; x0 += kThreads) {
          const int x = x0 + tid, h = min(x / quads, at_nh - 1), col = 4 * (x - x / quads * quads);
          float top = -INFINITY, sum = 0.f;
          float4 all4 = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
          for (int from = r0; from <= r1; from += fit) {
            const int n = min(fit, r1 - from + 1);
            __syncthreads();
#pragma unroll 1
            for (int y = tid; y < n * at_nh; y += kThreads) {
              const int r = from + y / at_nh;
              part[y] = __ldcg(&work.stats[(2 * r + (r == r0)) * kMaxHeads + y % at_nh]);
            }
            __syncthreads();
            float next = top;
#pragma unroll 4
            for (int r = 0; r < n; ++r) next = fmaxf(next, part[r * at_nh + h].x);
            const float keep = share(make_float2(top, 0.f), next);
            sum *= keep;
            all4 = add(make_float4(0.f, 0.f, 0.f, 0.f), keep, all4);
            top = next;
            // (the loads do not wait for the maxima)
#pragma unroll 16
            for (int r = 0; r < n; ++r) {
              const int slot = (2 * (from + r) + (from + r == r0)) * kMaxHeads + h;
              const float4 y = __ldcg(reinterpret_cast<const float4*>(work.sums + (long long)slot * attn::kMaxDim + col));
              const float2 st = part[r * at_nh + h];
              const float f = share(st, top);
              sum = fmaf(f, st.y, sum);
              all4 = add(all4, f, y);
            }
          }
          if (x < at_nh * quads) put(h, col, all4, top, sum);
        }
      }
    }
    if (!more) break;
  }
}

namespace {

int resident(int sms) { return sms * kCtas; }

// Workspace: [256 B, a caller's status words][partial sums][their maxima and sums][counters].  The places do not depend on the
// call, so that the counters are zero whatever call came before.
struct Layout {
  size_t stats, counters, total;
};
Layout layout(int B, int Hq, int Hkv, int sms) {
  const int G = Hq / Hkv, groups = (G + kMaxHeads - 1) / kMaxHeads;
  const size_t slots = 2 * (size_t)resident(sms) * kMaxHeads;
  Layout l;
  l.stats = 256 + slots * attn::kMaxDim * 4;
  l.counters = l.stats + slots * 8;
  l.total = l.counters + ((size_t)B * Hkv * groups * 4 + 255) / 256 * 256;
  return l;
}

template <int NT, int NC, bool E4M3>
cudaError_t launch_step(const StepArgs& a, int groups, int heads, unsigned grid, Work w, int* err, cudaStream_t st) {
  constexpr int kSmem = Ring<NT, NC, E4M3>::kSmem;
  const cudaError_t e = set_smem_limit_once<gdn_attn_step_kernel<NT, NC, E4M3>>(kSmem);
  if (e != cudaSuccess) return e;
  gdn_attn_step_kernel<NT, NC, E4M3>
      <<<grid, kThreads, kSmem, st>>>(a, groups, heads, a.scale * attn::kLog2e, a.d % 16 == 0, w, err);
  return cudaGetLastError();
}

}  // namespace

size_t attn_step_workspace(int B, int Hq, int Hkv, int d) {
  const int sms = device_sms();
  return layout(B, Hq, Hkv, sms > 0 ? sms : 256).total;  // (without a device: enough for any)
}

cudaError_t launch_attn_step(const StepArgs& a, bool e4m3, void* ws, int* status, cudaStream_t st) {
  const int sms = device_sms();
  if (sms == 0) return cudaErrorNoDevice;
  const int G = a.Hq / a.Hkv, groups = (G + kMaxHeads - 1) / kMaxHeads, heads = (G + groups - 1) / groups;
  if ((long long)a.B * a.Hkv * groups > 0x3fffffffLL) return cudaErrorInvalidValue;
  const Layout l = layout(a.B, a.Hq, a.Hkv, sms);
  unsigned char* p = static_cast<unsigned char*>(ws);
  Work w = {reinterpret_cast<float*>(p + 256), reinterpret_cast<float2*>(p + l.stats),
            reinterpret_cast<int*>(p + l.counters)};
  const unsigned grid = (unsigned)resident(sms);
  auto run = [&](auto nt, auto e) {
    constexpr int NT = decltype(nt)::value;
    constexpr bool E4M3 = decltype(e)::value;
    switch ((a.d + 31) / 32) {
      case 1: return launch_step<NT, 1, E4M3>(a, groups, heads, grid, w, status, st);
      case 2: return launch_step<NT, 2, E4M3>(a, groups, heads, grid, w, status, st);
      case 3: return launch_step<NT, 3, E4M3>(a, groups, heads, grid, w, status, st);
      default: return launch_step<NT, 4, E4M3>(a, groups, heads, grid, w, status, st);
    }
  };
  using One = std::integral_constant<int, 1>;
  using Two = std::integral_constant<int, 2>;
  if (heads <= 8) return e4m3 ? run(One(), std::true_type()) : run(One(), std::false_type());
  return e4m3 ? run(Two(), std::true_type()) : run(Two(), std::false_type());
}

}  // namespace gdn
