// The kernels of the chunked selective scan (gdn_ssm_chunk.cuh has the mathematics); one translation
// unit per state width instantiates them.
#pragma once

#include "gdn_ssm_chunk.cuh"

namespace gdn {
namespace ssm {

constexpr int kBars = 15;
constexpr int kSegStages = 3;  // of the pass of the sums

// What both kernels set up: shared memory (from a 1024-byte boundary, as the swizzled tiles want), TMEM, barriers.
struct Frame {
  unsigned char* sm;
  uint32_t sb;  // shared-window address of sm
  uint64_t* bars;
  uint32_t* tmem_slot;
  volatile int* abort_flag;
  SsmDecay* lend;  // [4 buffers][heads]: e^{L_last}
  float* gaps;     // [heads][4 blocks]: Tables::gap
  float* tabs;     // [heads][L, K, far, w, e]
};
template <class C>
__device__ __forceinline__ Frame make_frame(unsigned char* raw) {
  Frame f;
  f.sm = raw;
  f.sb = smem_u32(raw);
  f.bars = reinterpret_cast<uint64_t*>(f.sm + C::kOffBar);
  f.tmem_slot = reinterpret_cast<uint32_t*>(f.bars + kBars);
  f.abort_flag = reinterpret_cast<volatile int*>(f.tmem_slot + 1);
  f.lend = reinterpret_cast<SsmDecay*>(f.tmem_slot + 2);
  f.gaps = reinterpret_cast<float*>(f.bars) + 48;  // past kBars barriers, two words and eight decays
  f.tabs = reinterpret_cast<float*>(f.sm + C::kOffTab);
  return f;
}

// B and x of the chunk that starts at token t into a stage.
template <int DK, int PB, class C>
__device__ __forceinline__ void load_stage(const Frame& f, int stage, const CUtensorMap* tm_b, const CUtensorMap* tm_x,
                                           int hk, int h0, int dv, int t, uint64_t* bar) {
  unsigned char* dst = f.sm + stage * C::kStage;
  tc::mbar_arrive_expect_tx(bar, C::kStage);
#pragma unroll
  for (int i = 0; i < C::kNB; ++i) tc::tma_load_2d(dst + C::kOffB + i * 16384, tm_b, hk * DK + 64 * i, t, bar);
#pragma unroll
  for (int i = 0; i < C::kXB; ++i)
    tc::tma_load_2d(dst + C::kOffX + i * 16384, tm_x, PB == 64 ? (h0 + i) * dv : h0 * dv + 64 * i, t, bar);
}

// A segment's sum in the workspace is laid out by threads, kSC values of each of the 512 workers, float4 by float4,
// so that a warp's access is one run of 512 bytes.
template <class C>
__device__ __forceinline__ size_t seg_at(int slot, int nhb, int hb, int tid) {
  return (((size_t)slot * nhb + hb) * (C::kSC / 4) * (32 * kWorkers) + tid) * 4;
}

// The state of the CTA's heads between memory (rows of DK values, the heads one after the other) and the workers'
// registers, by way of a piece of shared memory of each warp's own (in the state operand's place): its 32 rows, up to
// 16 columns at a time, 16-byte pieces XORed with the row so that both orders are free of bank conflicts.
template <int DK, int PB, int HPC, bool kStore>
__device__ __forceinline__ void move_state(unsigned char* place, float* mem, int dv, const Worker& me,
                                           float (&st)[DK / 4]) {
  constexpr int kSC = DK / 4, kPart = kSC < 16 ? kSC : 16, kPc = kPart / 4, kParts = kSC / kPart;
  const int row0 = 32 * me.q4, p0 = PB == 64 ? row0 & 63 : row0;
  if (row0 >= PB * HPC || p0 >= dv) return;
  unsigned char* buf = place + (me.cg * (PB * HPC / 32) + me.q4) * (32 * kPart * 4);
  auto at = [&](int row, int piece) {
    return reinterpret_cast<float4*>(buf + (row * kPc + (piece ^ ((row / (8 / kPc)) & (kPc - 1)))) * 16);
  };
  float4* m = reinterpret_cast<float4*>(mem + (size_t)((HPC == 2 ? row0 >> 6 : 0) * dv + p0) * DK + kSC * me.cg);
  auto out_at = [&](int part, int i) {  // memory order: lane's piece i of a part
    const int e = me.lane + 32 * i;
    return m + (e / kPc) * (DK / 4) + part * kPc + e % kPc;
  };
  float4 v[kParts][kPc];
  if (!kStore) {
#pragma unroll
    for (int h = 0; h < kParts; ++h)
#pragma unroll
      for (int i = 0; i < kPc; ++i) v[h][i] = *out_at(h, i);
  }
#pragma unroll
  for (int h = 0; h < kParts; ++h) {
#pragma unroll
    for (int i = 0; i < kPc; ++i) {
      const float* q = st + h * kPart + 4 * i;
      if (kStore) *at(me.lane, i) = make_float4(q[0], q[1], q[2], q[3]);
      else *at((me.lane + 32 * i) / kPc, (me.lane + 32 * i) % kPc) = v[h][i];
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kPc; ++i) {
      if (kStore) {
        *out_at(h, i) = *at((me.lane + 32 * i) / kPc, (me.lane + 32 * i) % kPc);
      } else {
        const float4 t = *at(me.lane, i);
        float* q = st + h * kPart + 4 * i;
        q[0] = t.x; q[1] = t.y; q[2] = t.z; q[3] = t.w;
      }
    }
    __syncwarp();
  }
}

// Outputs (and the final state of a sequence's last segment) of one segment and head block.
// grid: segments x head blocks, the head blocks of a segment side by side (they read the same B and C).
template <int DK, int PB, int HPC>
__global__ void __launch_bounds__(kThreads, 1)
gdn_ssm_chunk_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_b,
                     const __grid_constant__ CUtensorMap tm_c, const __grid_constant__ CUtensorMap tm_z,
                     const __grid_constant__ CUtensorMap tm_o, const SsmArgs a, const Segs g,
                     const float* seg_state, const float* seg_decay, const float* init, const float* kept, float* fin,
                     int* __restrict__ err) {
  using C = Cfg<DK, PB, HPC>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const Frame f = make_frame<C>(smem_raw);
  // Completed by the MMAs, once a chunk each: scores; (w x)^T B of half 0 and C S^T; (w x)^T B of half 1; y.  By
  // copies: the two stages, C, the gate's tile.  By the worker warps: the first operands of a chunk (the state, w x),
  // the second (w x), the gate read, y read, the outputs out of the x tile, y scaled and M.  By the table warp: a
  // chunk's tables made and its stage loaded.  Every waiter waits for every phase in turn, and no phase after it can
  // end before it has looked (a parity only names the last phase that ended): what leads to the next one waits for
  // the waiter.
  uint64_t *b_sc = f.bars, *b_in = f.bars + 1, *b_d1 = f.bars + 2, *b_y = f.bars + 3, *b_st = f.bars + 4,
           *b_c = f.bars + 6, *b_z = f.bars + 7, *w_a = f.bars + 8, *w_b = f.bars + 9, *w_z = f.bars + 10,
           *w_y = f.bars + 11, *w_s = f.bars + 12, *b_tab = f.bars + 13, *w_m = f.bars + 14;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp == kAllocWarp) {
    tc::tmem_alloc(f.tmem_slot, kTmemCols);
    tc::tmem_relinquish();
  }
  const int nhb = a.Hv / HPC, seg = blockIdx.x / nhb;
  const int h0 = (blockIdx.x - seg * nhb) * HPC;
  const int hk = h0 / (a.Hv / a.Hk);
  Seg s;
  const bool live = find_seg(g, seg, s);
  if (!live) s.t0 = s.t1 = 0, s.b = 0, s.p = 0, s.bos = 0, s.slot = 0, s.first = s.last = false;
  const int ntok = s.t1 - s.t0, nc = (ntok + kQ - 1) / kQ;
  const long long tok0 = s.bos + s.t0;
  auto load = [&](int c) {
    load_stage<DK, PB, C>(f, c & 1, &tm_b, &tm_x, hk, h0, a.dv, (int)(tok0 + (long long)c * kQ), &b_st[c & 1]);
  };
  auto load_c = [&](int c) {
    const int t = (int)(tok0 + (long long)c * kQ);
    tc::mbar_arrive_expect_tx(b_c, C::kNB * 16384);
#pragma unroll
    for (int i = 0; i < C::kNB; ++i) tc::tma_load_2d(f.sm + C::kOffC + i * 16384, &tm_c, hk * DK + 64 * i, t, b_c);
  };
  if (warp == kIssueWarp && lane == 0) {  // the inputs are there whatever runs before: the first tiles at once
    for (int i = 0; i < kBars; ++i) tc::mbar_init(&f.bars[i], i >= 8 && i != 13 ? kWorkers : 1);
    tc::fence_mbar_init();
    *f.abort_flag = 0;
    if (nc > 0) {
      load(0);
      load_c(0);
      if (nc > 1) load(1);
    }
    if (g.cu != nullptr && h0 == 0 && live && s.first) {
      const int lo = g.cu[s.b], hi = g.cu[s.b + 1];
      if (lo < 0 || hi < lo || hi > g.T || (s.b == 0 && lo != 0) || (s.b == g.B - 1 && hi != g.T)) atomicOr(err, 8);
    }
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *f.tmem_slot;
  const bool gate = a.z != nullptr;
  int gave_up = 0;  // the status bit of the wait that this warp gave up
  auto wait1 = [&](uint64_t* bar, uint32_t par, int bit) {
    const bool done = tc::mbar_wait(bar, par, g.polls);
    if (!done) gave_up = bit;
    return done;
  };
  // A whole warp, together and of one mind after it.  (With the limit from the parameters in these loops 32 ragged
  // prompts take 562 us, with the constant 553.)
  auto wait = [&](uint64_t* bar, uint32_t par, int bit) {
    const bool done = __all_sync(0xffffffffu, tc::mbar_wait(bar, par, kMaxPolls)) != 0;
    if (!done) gave_up = bit;
    return done;
  };

  // The same, where the phase was looked at before.
  auto settle = [&](uint32_t seen, uint64_t* bar, uint32_t par, int bit) {
    const bool done = __all_sync(0xffffffffu, seen) != 0;
    asm volatile("" ::: "memory");
    return done || wait(bar, par, bit);
  };

  if (warp == kIssueWarp) {
    // ================= copies and MMAs: one thread =================
    auto load_z = [&](int c) {
      const int t = (int)(tok0 + (long long)c * kQ);
      tc::mbar_arrive_expect_tx(b_z, C::kXB * 16384);
#pragma unroll
      for (int i = 0; i < C::kXB; ++i)
        tc::tma_load_2d(f.sm + C::kOffZ + i * 16384, &tm_z, PB == 64 ? (h0 + i) * a.dv : h0 * a.dv + 64 * i, t, b_z);
    };
    const uint64_t c_kmajor = tc::sdesc(f.sb + C::kOffC, 16, 1024, tc::kSw128);
    // scores of chunk c: C_i . B_j over the chunk's tokens, once both tiles are in
    auto scores = [&](int c) {
      if (!wait1(&b_st[c & 1], (uint32_t)((c >> 1) & 1), 2) || !wait1(b_c, (uint32_t)(c & 1), 2)) return false;
      constexpr uint32_t kId = tc::idesc_bf16(128, 128, 0, 0);
      const uint64_t bd = tc::sdesc(f.sb + (c & 1) * C::kStage + C::kOffB, 16, 1024, tc::kSw128);
#pragma unroll
      for (int ks = 0; ks < DK / 16; ++ks) {
        const uint64_t off = (uint64_t)(((ks >> 2) * 16384 + (ks & 3) * 32) >> 4);
        tc::mma_bf16(tmem + kColSc, c_kmajor + off, bd + off, kId, ks > 0);
      }
      tc::commit(b_sc);
      return true;
    };
    if (lane == 0 && nc > 0) {
      bool ok = scores(0);
      for (int c = 0; ok && c < nc; ++c) {
        const uint32_t par = (uint32_t)(c & 1);
        const uint32_t stage = f.sb + (c & 1) * C::kStage;
        if (!(ok = wait1(w_a, par, 1))) break;
        tc::fence_after();
        issue_state<DK>(tmem + kColDs, tmem + kColXw, stage + C::kOffB, 0, true);
        if (c > 0) {  // the chunk before's y has been read
          if (!(ok = wait1(w_y, par ^ 1u, 1))) break;
          tc::fence_after();
        }
        {
          constexpr uint32_t kId = tc::idesc_bf16(128, C::kRows, 0, 0);
          const uint64_t bd = tc::sdesc(f.sb + C::kOffS, 16, 1024, tc::kSw128);
#pragma unroll
          for (int ks = 0; ks < DK / 16; ++ks)
            tc::mma_bf16(tmem + kColY, c_kmajor + (uint64_t)(((ks >> 2) * 16384 + (ks & 3) * 32) >> 4),
                         bd + (uint64_t)(((ks >> 2) * (C::kRows * 128) + (ks & 3) * 32) >> 4), kId, ks > 0);
          tc::commit(b_in);
        }
        if (C::kOwnGate && gate) {
          if (c > 0 && !(ok = wait1(w_z, par ^ 1u, 1))) break;
          load_z(c);
        }
        if (c + 1 < nc || (!C::kOwnGate && gate)) {
          if (!(ok = wait1(b_in, par, 1))) break;
          if (!C::kOwnGate && gate) load_z(c);  // over the state operand
          if (c + 1 < nc) load_c(c + 1);
          if (c > 0 && c + 1 < nc) {  // the stage of the chunk before
            if (!(ok = wait1(w_s, par ^ 1u, 1))) break;
            load(c + 1);
          }
        }
        if (!(ok = wait1(w_b, par, 1))) break;
        tc::fence_after();
        issue_state<DK>(tmem + kColDs, tmem + kColXw, stage + C::kOffB, 1, false);
        tc::commit(b_d1);
        if (!(ok = wait1(w_m, par, 1))) break;
        tc::fence_after();
        {
          constexpr uint32_t kId = tc::idesc_bf16(128, PB, 0, 1);
#pragma unroll
          for (int hh = 0; hh < HPC; ++hh) {
            const uint64_t xd = tc::sdesc(stage + C::kOffX + hh * 16384, 16384, 1024, tc::kSw128);
#pragma unroll
            for (int ks = 0; ks < kQ / 16; ++ks)
              tc::mma_f16_ta(tmem + kColY + hh * PB, tmem + kColSc + 16 * ks + 8 * hh,
                             xd + (uint64_t)((ks * 2048) >> 4), kId, 1u);
          }
          tc::commit(b_y);
        }
        if (c + 1 < nc) {  // the next scores take M's place, once M x is done
          if (!(ok = wait1(b_y, par, 1))) break;
          ok = scores(c + 1);
        }
      }
    }
    __syncwarp();
  } else if (warp == kTableWarp) {
    // ================= tables, a chunk ahead =================
    float a_log2[HPC], bias[HPC];
    uint32_t raw[HPC][4];
#pragma unroll
    for (int hh = 0; hh < HPC; ++hh) {
      a_log2[hh] = a.A[h0 + hh] * 1.4426950408889634f;
      bias[hh] = ssm_bias(a, h0 + hh);
      if (nc > 0) load_dt(a, tok0, ntok, h0 + hh, lane, raw[hh]);
    }
    for (int c = 0; c < nc; ++c) {
      Tables t[HPC];
#pragma unroll
      for (int hh = 0; hh < HPC; ++hh) {
        float d[4];
        to_steps(a, ntok - c * kQ, bias[hh], lane, raw[hh], d);
        if (c + 1 < nc) load_dt(a, tok0 + (long long)(c + 1) * kQ, ntok - (c + 1) * kQ, h0 + hh, lane, raw[hh]);
        t[hh] = make_tables(d, a_log2[hh], lane);
      }
      if (!wait(&b_st[c & 1], (uint32_t)((c >> 1) & 1), 2)) break;
      // the tables of chunk c - 1 were read up to its M (the decays, used after it, have four places)
      if (c > 0 && !wait(w_m, (uint32_t)((c - 1) & 1), 1)) break;
#pragma unroll
      for (int hh = 0; hh < HPC; ++hh) {
        float4* tab = reinterpret_cast<float4*>(f.tabs + hh * 5 * kQ);
        tab[lane] = t[hh].L;
        tab[32 + lane] = t[hh].K;
        tab[64 + lane] = t[hh].far;
        tab[96 + lane] = t[hh].w;
        tab[128 + lane] = t[hh].e;
        if ((lane & 7) == 0) reinterpret_cast<float2*>(f.gaps)[hh * 4 + (lane >> 3)] = t[hh].gap;
        if (lane == 0) f.lend[(c & 3) * HPC + hh] = ssm_decay(t[hh].end * 0.6931471805599453f);
      }
      __syncwarp();
      if (lane == 0) arrive(b_tab);
      // into L2, since their places in shared memory are free only late: the next gate, x and B
      if (lane == 0) {
        const int t = (int)(tok0 + (long long)c * kQ);
#pragma unroll
        for (int i = 0; i < C::kXB; ++i) {
          const int col = PB == 64 ? (h0 + i) * a.dv : h0 * a.dv + 64 * i;
          if (gate && c == 0) tma_prefetch_l2_2d(&tm_z, col, t);
          if (gate && c + 1 < nc) tma_prefetch_l2_2d(&tm_z, col, t + kQ);
          if (c > 0 && c + 1 < nc) tma_prefetch_l2_2d(&tm_x, col, t + kQ);
        }
        if (c > 0 && c + 1 < nc)
#pragma unroll
          for (int i = 0; i < C::kNB; ++i) tma_prefetch_l2_2d(&tm_b, hk * DK + 64 * i, t + kQ);
      }
      __syncwarp();
    }
  } else if (warp < kWorkers) {
    // ================= workers =================
    auto lanes_of = [&](const Worker& me) { return tmem + ((uint32_t)(32 * me.q4) << 16); };  // its TMEM lanes
    auto head_of = [](int row) { return HPC == 2 ? row >> 6 : 0; };                            // a state row's head
    float st[C::kSC];  // this thread's state: its row (head, p), columns kSC cg ..
#pragma unroll
    for (int i = 0; i < C::kSC; ++i) st[i] = 0.f;
    const size_t st_at = ((size_t)s.b * a.Hv + h0) * a.dv * DK;
    asm volatile("griddepcontrol.wait;\n" ::: "memory");  // the segments' sums
    if (live && init != nullptr) {  // where the final state replaces it, the later segments' copy of it
      const float* from = kept != nullptr && !(s.first && s.last) ? kept : init;
      move_state<DK, PB, HPC, false>(f.sm + C::kOffS, const_cast<float*>(from) + st_at, a.dv, worker(), st);
      asm volatile("bar.sync 1, %0;\n" ::"n"(32 * kWorkers) : "memory");  // before the state operand
    }
    // the sums of the segments before: one by one where they are few, or joined into one
    const int i0 = g.joined ? s.slot : s.slot - s.p, i1 = s.slot + (g.joined && s.p > 0 ? 1 : 0);
    const int my_p = PB == 64 ? tid & 63 : tid & 127;
    // half of a sum's values are on their way while the other half is added
    if (live && (tid & 127) < C::kRows && my_p < a.dv && i0 < i1) {
      constexpr int kH = C::kSC / 8;
      auto fetch = [&](int i, int hf, float4 (&v)[kH]) {
        const float4* e = reinterpret_cast<const float4*>(seg_state + seg_at<C>(i, nhb, h0 / HPC, tid));
#pragma unroll
        for (int u = 0; u < kH; ++u) v[u] = e[(hf * kH + u) * 32 * kWorkers];
      };
      auto add = [&](const SsmDecay& d, int hf, const float4 (&v)[kH]) {
#pragma unroll
        for (int u = 0; u < kH; ++u) {
          float* q = st + 4 * (hf * kH + u);
          q[0] = ssm_decayed(d, q[0], v[u].x);
          q[1] = ssm_decayed(d, q[1], v[u].y);
          q[2] = ssm_decayed(d, q[2], v[u].z);
          q[3] = ssm_decayed(d, q[3], v[u].w);
        }
      };
      const float* dec = seg_decay + h0 + head_of(tid & 127);
      float4 lo[kH], hi[kH];
      float l = dec[(size_t)i0 * a.Hv];
      fetch(i0, 0, lo);
      for (int i = i0; i < i1; ++i) {
        fetch(i, 1, hi);
        const SsmDecay d = ssm_decay(l * 0.6931471805599453f);
        if (i + 1 < i1) l = dec[(size_t)(i + 1) * a.Hv];
        add(d, 0, lo);
        if (i + 1 < i1) fetch(i + 1, 0, lo);
        add(d, 1, hi);
      }
    }
    // a warp's outputs: tokens 32 q4 .. + 31, columns kYC cg .., worked on by rows in the warp's own part of the x tile
    // and stored from there in memory order (kP 16-byte pieces a token)
    constexpr int kP = C::kYC / 8;
    struct Cols {
      int h, p;             // head and its first column
      uint32_t off, piece;  // offset of the tile's 64-wide block, first 16-byte piece in its rows
      int quad;             // named barrier of the warps that share 32 tokens of the block
    };
    auto cols_of = [](const Worker& me) {
      const int yc = C::kYC * me.cg;
      return Cols{HPC == 2 ? yc >> 6 : 0, PB == 64 ? yc & 63 : yc, (uint32_t)(yc >> 6) * 16384,
                  (uint32_t)(yc & 63) >> 3, 2 + 4 * (yc >> 6) + me.q4};
    };
    float skip = 0.f;
    {
      const Cols y = cols_of(worker());
      if (a.D != nullptr && y.p < a.dv) skip = a.D[h0 + y.h];
    }
    bool ok = true;
    // The first operands of chunk c: the state, and w x of its first 64 tokens.
    auto first_operands = [&](int c, uint32_t seen) {
      const Worker me = worker();
      unsigned char* stage = f.sm + (c & 1) * C::kStage;
      const int n = min(kQ, ntok - c * kQ);
      if (!settle(seen, b_tab, (uint32_t)(c & 1), 1)) return false;
      if (n < kQ) {  // rows of the sequence after this one: zeros, so that no value of theirs meets a zero weight
        const int rows = kQ - n;
        for (int e = 128 * me.cg + me.row; e < rows * 8 * (C::kNB + C::kXB); e += 32 * kWorkers)
          *reinterpret_cast<uint4*>(stage + (e / (rows * 8)) * 16384 + (n * 8 + e % (rows * 8)) * 16) =
              make_uint4(0, 0, 0, 0);
        __syncwarp();
        asm volatile("bar.sync 1, %0;\n" ::"n"(32 * kWorkers) : "memory");
      }
      if (!C::kOwnGate && gate && c > 0) {  // the gate there is read
        if (!wait(w_z, (uint32_t)((c - 1) & 1), 1)) return false;
      }
      XwTiles xw;
      if (32 * me.q4 < C::kRows)
        load_xw(xw, stage + C::kOffX, f.tabs + head_of(me.row) * 5 * kQ + 3 * kQ, me.lane, 32 * me.q4, 16 * me.cg);
      if (me.row < C::kRows) {
#pragma unroll
        for (int i = 0; i < C::kSC; i += 8) {
          const int col = C::kSC * me.cg + i;
          *reinterpret_cast<uint4*>(f.sm + C::kOffS + (col >> 6) * (C::kRows * 128) +
                                    tc::sw128((uint32_t)me.row, (uint32_t)(col & 63) >> 3)) =
              make_uint4(pack_bf16(st[i], st[i + 1]), pack_bf16(st[i + 2], st[i + 3]), pack_bf16(st[i + 4], st[i + 5]),
                         pack_bf16(st[i + 6], st[i + 7]));
        }
      }
      if (32 * me.q4 < C::kRows) split_xw(xw, lanes_of(me) + kColXw + 8 * me.cg);
      tmem_st_wait();
      tc::fence_proxy_async();
      tc::fence_before();
      __syncwarp();
      if (me.lane == 0) arrive(w_a);
      return true;
    };
    if (nc > 0) ok = first_operands(0, 0);
    uint32_t seen_in = 0;
    for (int c = 0; ok && c < nc; ++c) {
      const uint32_t par = (uint32_t)(c & 1);
      unsigned char* xt = f.sm + (c & 1) * C::kStage + C::kOffX;

      // ---- w x of the other 64 tokens ------------------------------------------------------------------
      uint32_t seen_sc;
      {
        const Worker me = worker();
        XwTiles xw;
        if (32 * me.q4 < C::kRows)
          load_xw(xw, xt, f.tabs + head_of(me.row) * 5 * kQ + 3 * kQ, me.lane, 32 * me.q4, 64 + 16 * me.cg);
        if (!(ok = settle(seen_in, b_in, par, 1))) break;  // (w x)^T B of the first 64 and C S^T
        tc::fence_after();
        seen_sc = peek(b_sc, par);
        if (32 * me.q4 < C::kRows) split_xw(xw, lanes_of(me) + kColXw + 8 * me.cg);
        tmem_st_wait();
        tc::fence_before();
        bulk_wait_read();  // the chunk before's outputs have left its x tile
        __syncwarp();
        if (me.lane == 0) {
          arrive(w_b);
          if (c > 0) arrive(w_s);
        }
      }
      // ---- y = e^{L_i} (C S^T), in place ---------------------------------------------------------------
      {
        const Worker me = worker();
        const uint32_t at = lanes_of(me) + kColY + C::kYC * me.cg;
        const float e = f.tabs[cols_of(me).h * 5 * kQ + 4 * kQ + me.row];
#pragma unroll
        for (int i0 = 0; i0 < C::kYC; i0 += 16) {
          float y[16];
          tc::tmem_ld16(at + i0, y);
          uint32_t u[16];
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const float2 v = mul2(make_float2(y[i], y[i + 1]), make_float2(e, e));
            u[i] = __float_as_uint(v.x);
            u[i + 1] = __float_as_uint(v.y);
          }
          tmem_st16_nowait(at + i0, u);
        }
      }
      // ---- M from the scores, in their place: eight columns a head of each 16 ------------------------
      if (!(ok = settle(seen_sc, b_sc, par, 1))) break;
      tc::fence_after();
      {
        const Worker me = worker();
        const uint32_t col = lanes_of(me) + kColSc + 32 * me.cg;
        uint32_t m[8];
        if (me.cg <= me.q4) {
          float lis[HPC];
#pragma unroll
          for (int hh = 0; hh < HPC; ++hh) {
            lis[hh] = f.tabs[hh * 5 * kQ + me.row];
            if (me.cg + 1 < me.q4) lis[hh] += f.gaps[(hh * 4 + me.q4) * 2 + me.cg];  // blocks between
          }
#pragma unroll 1
          for (int j0 = 0; j0 < 32; j0 += 16) {
            float sc[16];
            tc::tmem_ld16(col + j0, sc);
            const int upto = me.cg == me.q4 ? me.lane - j0 : 32;  // this token's last column
#pragma unroll
            for (int hh = 0; hh < HPC; ++hh) {
              const float* th = f.tabs + hh * 5 * kQ;
              const float li = lis[hh];
              const float* tk = th + (me.cg == me.q4 ? kQ : 2 * kQ);
              const float2 minus = make_float2(-1.f, -1.f), l2 = make_float2(li, li);
#pragma unroll
              for (int j = 0; j < 16; j += 4) {
                const float4 k4 = *reinterpret_cast<const float4*>(tk + 32 * me.cg + j0 + j);
                const float2 e0 = fma2(make_float2(k4.x, k4.y), minus, l2);
                const float2 e1 = fma2(make_float2(k4.z, k4.w), minus, l2);
                float2 u = mul2(make_float2(sc[j], sc[j + 1]), make_float2(ex2_approx(e0.x), ex2_approx(e0.y)));
                float2 v = mul2(make_float2(sc[j + 2], sc[j + 3]), make_float2(ex2_approx(e1.x), ex2_approx(e1.y)));
                u.x = j <= upto ? u.x : 0.f;
                u.y = j + 1 <= upto ? u.y : 0.f;
                v.x = j + 2 <= upto ? v.x : 0.f;
                v.y = j + 3 <= upto ? v.y : 0.f;
                m[j / 2] = pack_bf16(u.x, u.y);
                m[j / 2 + 1] = pack_bf16(v.x, v.y);
              }
              if (!a.softplus) turn_signs(m, th + 3 * kQ + 32 * me.cg + j0);
              tmem_st8_nowait(col + j0 + 8 * hh, m);
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) m[j] = 0u;
#pragma unroll
          for (int hh = 0; hh < HPC; ++hh) {
            tmem_st8_nowait(col + 8 * hh, m);
            tmem_st8_nowait(col + 16 + 8 * hh, m);
          }
        }
      }
      tmem_st_wait();
      tc::fence_before();
      __syncwarp();
      if (lane == 0) arrive(w_m);
      // Some of the gate through silu while the state's product runs: what the registers have room for (32 ragged
      // prompts: 587 us with none, 560 with eight columns, 595 with sixteen).
      constexpr int kEarly = C::kOwnGate ? kP / 4 : 0;
      float2 ge[kEarly + 1][4];
      if (C::kOwnGate && gate) {
        if (!(ok = wait(b_z, par, 2))) break;
        const Worker me = worker();
        const Cols cols = cols_of(me);
#pragma unroll
        for (int i = 0; i < kEarly; ++i) {
          widen8(above_minus_inf(*reinterpret_cast<const uint4*>(f.sm + C::kOffZ + cols.off +
                                                                 tc::sw128((uint32_t)me.row, cols.piece + i))),
                 ge[i]);
#pragma unroll
          for (int u = 0; u < 4; ++u) ge[i][u] = silu2_above(ge[i][u]);
        }
      }
      uint4 zr[kP];
      if (!C::kOwnGate && gate) {  // the gate, before the next state takes its place
        if (!(ok = wait(b_z, par, 2))) break;
        const Worker me = worker();
        const Cols cols = cols_of(me);
#pragma unroll
        for (int i = 0; i < kP; ++i)
          zr[i] = *reinterpret_cast<const uint4*>(f.sm + C::kOffZ + cols.off +
                                                  tc::sw128((uint32_t)me.row, cols.piece + i));
        __syncwarp();
        if (me.lane == 0) arrive(w_z);
      }
      // ---- S = e^{L_last} S + the chunk's sum ---------------------------------------------------------
      const uint32_t seen_tab = peek(b_tab, par ^ 1u);
      if (!(ok = wait(b_d1, par, 1))) break;
      tc::fence_after();
      {
        float ds[C::kSC];  // (in two halves it spares spills and still costs 2% more, for a second wait)
        const Worker me = worker();
        tmem_load<C::kSC>(lanes_of(me) + kColDs + C::kSC * me.cg, ds);
        const SsmDecay decay = f.lend[(c & 3) * HPC + head_of(me.row)];
#pragma unroll
        for (int i = 0; i < C::kSC; i += 2) {
          const float2 v = make_float2(st[i], st[i + 1]);
          const float2 r = fma2(make_float2(decay.keep, decay.keep), v,
                                fma2(make_float2(decay.more, decay.more), v, make_float2(ds[i], ds[i + 1])));
          st[i] = r.x;
          st[i + 1] = r.y;
        }
      }
      if (c + 1 < nc && !(ok = first_operands(c + 1, seen_tab))) break;
      // ---- outputs, by way of the warp's own part of the x tile -----------------------------------------
      if (!(ok = wait(b_y, par, 1))) break;
      tc::fence_after();
      {
        const Worker me = worker();
        const Cols cols = cols_of(me);
        unsigned char* yt = xt + cols.off;
        const int n = min(kQ, ntok - c * kQ);
        float y[C::kYC];
        tmem_load<C::kYC>(lanes_of(me) + kColY + C::kYC * me.cg, y);
        tc::fence_before();
        __syncwarp();
        if (me.lane == 0) arrive(w_y);
#pragma unroll
        for (int i = 0; i < kP; ++i) {  // eight columns of this thread's own row at a time
          const uint32_t piece = tc::sw128((uint32_t)me.row, cols.piece + i);
          uint4* at = reinterpret_cast<uint4*>(yt + piece);
          float2 v[4], g4[4];
          widen8(*at, v);
          if (gate && i >= kEarly) {
            if (C::kOwnGate) zr[i] = *reinterpret_cast<const uint4*>(f.sm + C::kOffZ + cols.off + piece);
            widen8(above_minus_inf(zr[i]), g4);
          }
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            v[u] = fma2(v[u], make_float2(skip, skip), make_float2(y[8 * i + 2 * u], y[8 * i + 2 * u + 1]));
            if (gate) v[u] = mul2(v[u], i < kEarly ? ge[i < kEarly ? i : 0][u] : silu2_above(g4[u]));
          }
          *at = narrow8(v);
        }
        if (C::kOwnGate && gate) {
          __syncwarp();
          if (me.lane == 0) arrive(w_z);
        }
        seen_in = peek(b_in, par ^ 1u);
        // 32 whole tokens of 64 columns: one copy by the first of their warps
        if (a.dv >= 64 && 32 * me.q4 + 32 <= n) {
          tc::fence_proxy_async();
          asm volatile("bar.sync %0, %1;\n" ::"r"(cols.quad), "n"(32 * (64 / C::kYC)) : "memory");
          if (cols.piece == 0 && me.lane == 0) {
            tma_store_2d(&tm_o, smem_u32(yt) + 32 * me.q4 * 128, (h0 + cols.h) * a.dv + cols.p,
                         (int)(tok0 + (long long)c * kQ) + 32 * me.q4);
            bulk_commit();
          }
          __syncwarp();
        } else {
          __syncwarp();
          if (cols.p < a.dv) {
            const int mt = 32 * me.q4 + me.lane / kP, mp = me.lane % kP;  // token mt + (32 / kP) i, piece mp
            __nv_bfloat16* o =
                a.out + ((size_t)(tok0 + (long long)c * kQ) * a.Hv + h0 + cols.h) * a.dv + cols.p + 8 * mp;
#pragma unroll
            for (int i = 0; i < kP; ++i) {
              const int t = mt + (32 / kP) * i;
              if (t < n)
                *reinterpret_cast<uint4*>(o + (size_t)t * a.Hv * a.dv) =
                    *reinterpret_cast<const uint4*>(yt + tc::sw128((uint32_t)t, cols.piece + mp));
            }
          }
          tc::fence_proxy_async();
        }
      }
    }
    bulk_wait_read();
    if (!ok) {  // another warp may have passed the wait that this one gave up, and stand at a barrier between warps
      asm volatile("bar.arrive 1, %0;\n" ::"n"(32 * kWorkers) : "memory");
      asm volatile("bar.arrive %0, %1;\n" ::"r"(cols_of(worker()).quad), "n"(32 * (64 / C::kYC)) : "memory");
    }
    if (ok && fin != nullptr && live && s.last) {
      __syncwarp();
      // the state operand's place is free: C S^T is done, and the gate there read
      if (C::kOwnGate || !gate || nc == 0 || wait(w_z, (uint32_t)((nc - 1) & 1), 1))
        move_state<DK, PB, HPC, true>(f.sm + C::kOffS, fin + st_at, a.dv, worker(), st);
    }
  }
  const Worker at_end = worker();
  if (gave_up != 0 && at_end.lane == 0) {
    *f.abort_flag = 1;
    atomicOr(err, gave_up);
  }
  tc::fence_before();
  __syncthreads();
  if (*f.abort_flag) {  // let what is in flight land, bounded again
    if (at_end.row == 0 && at_end.cg == 0) {
      for (int i = 0; i < 8; ++i)
        for (uint32_t par = 0; par < 2; ++par) (void)tc::mbar_wait(&f.bars[i], par, 1u << 14);
    }
    __syncthreads();
  }
  if (4 * at_end.cg + at_end.q4 == kAllocWarp) {
    __syncwarp();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

// The sums of the segments before a sequence's last (from a zero state) and their decays in log2, and, where the final
// states will replace the initial ones, a copy of these.  Three stages of B and x: with two, a chunk's load (about
// 2,000 cycles) stood in the way of every chunk.  grid: segments x head blocks.
template <int DK, int PB, int HPC>
__global__ void __launch_bounds__(kThreads, 1)
gdn_ssm_segment_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_b,
                       const SsmArgs a, const Segs g, float* __restrict__ seg_state, float* __restrict__ seg_decay,
                       const float* __restrict__ init, float* __restrict__ kept, int* __restrict__ err) {
  using C = Cfg<DK, PB, HPC>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const Frame f = make_frame<C>(smem_raw);
  constexpr int kSC = C::kSC;
  static_assert(kSegStages * C::kStage <= C::kOffTab, "stages");
  // the sum; the stages loaded; w x written and tables made, for even and odd chunks
  uint64_t *b_d = f.bars, *b_st = f.bars + 1, *w_a = f.bars + 4, *b_tab = f.bars + 6;
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");  // what follows starts up beside this pass
  const int nhb = a.Hv / HPC, seg = blockIdx.x / nhb;
  Seg s;
  if (!find_seg(g, seg, s) || s.last) return;  // a last segment's sum is nobody's start
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp == kAllocWarp) {
    tc::tmem_alloc(f.tmem_slot, kTmemCols);
    tc::tmem_relinquish();
  }
  const int h0 = (blockIdx.x - seg * nhb) * HPC;
  const int hk = h0 / (a.Hv / a.Hk);
  const int nc = (s.t1 - s.t0) / kQ;  // whole chunks: only a last segment is ragged
  const long long tok0 = s.bos + s.t0;
  auto load = [&](int c) {
    load_stage<DK, PB, C>(f, c % kSegStages, &tm_b, &tm_x, hk, h0, a.dv, (int)(tok0 + (long long)c * kQ),
                          &b_st[c % kSegStages]);
  };
  if (warp == kIssueWarp && lane == 0) {
    for (int i = 0; i < kBars; ++i) tc::mbar_init(&f.bars[i], i == 4 || i == 5 ? kWorkers : 1);
    tc::fence_mbar_init();
    *f.abort_flag = 0;
    for (int c = 0; c < kSegStages && c < nc; ++c) load(c);
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *f.tmem_slot;
  int gave_up = 0;  // the status bit of the wait that this warp gave up
  auto wait1 = [&](uint64_t* bar, uint32_t par, int bit) {
    const bool done = tc::mbar_wait(bar, par, g.polls);
    if (!done) gave_up = bit;
    return done;
  };
  auto wait = [&](uint64_t* bar, uint32_t par, int bit) {  // a whole warp, together and of one mind after it
    const bool done = __all_sync(0xffffffffu, tc::mbar_wait(bar, par, g.polls)) != 0;
    if (!done) gave_up = bit;
    return done;
  };
  // TMEM: w x of a chunk (two halves of 96 columns) in two buffers, the sum between them
  constexpr uint32_t kSum = 288;
  auto xw_col = [](int c, int hf) { return (uint32_t)((c & 1) ? (hf ? 416 : 192) : (hf ? 96 : 0)); };

  if (warp == kIssueWarp) {
    if (lane == 0) {
      for (int c = 0; c < nc; ++c) {
        if (!wait1(&w_a[c & 1], (uint32_t)((c >> 1) & 1), 1)) break;  // w x of chunk c written, the sum of c - 1 read
        tc::fence_after();
        if (c > 0 && c + kSegStages - 1 < nc) load(c + kSegStages - 1);  // the stage of chunk c - 1
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
          issue_state<DK>(tmem + kSum, tmem + xw_col(c, hf), f.sb + (c % kSegStages) * C::kStage + C::kOffB, hf,
                          hf == 0);
        tc::commit(b_d);
      }
    }
    __syncwarp();
  } else if (warp >= kWorkers) {
    // even and odd chunks' tables
    const int odd = warp == (kTableWarp + 1);
    float a_log2[HPC], bias[HPC], total[HPC];
    uint32_t raw[HPC][4];
#pragma unroll
    for (int hh = 0; hh < HPC; ++hh) {
      a_log2[hh] = a.A[h0 + hh] * 1.4426950408889634f;
      bias[hh] = ssm_bias(a, h0 + hh);
      total[hh] = 0.f;
      if (odd < nc) load_dt(a, tok0 + odd * kQ, kQ, h0 + hh, lane, raw[hh]);
    }
    for (int c = odd; c < nc; c += 2) {
      // the tables of chunk c - 2 were read before its operands were announced
      if (c > 1 && !wait(&w_a[odd], (uint32_t)(((c - 2) >> 1) & 1), 1)) break;
#pragma unroll
      for (int hh = 0; hh < HPC; ++hh) {
        float d[4];
        to_steps(a, kQ, bias[hh], lane, raw[hh], d);
        if (c + 2 < nc) load_dt(a, tok0 + (long long)(c + 2) * kQ, kQ, h0 + hh, lane, raw[hh]);
        const Tables t = make_tables(d, a_log2[hh], lane);
        reinterpret_cast<float4*>(f.tabs + (odd * HPC + hh) * kQ)[lane] = t.w;
        total[hh] += t.end;
        if (lane == 0) f.lend[odd * HPC + hh] = ssm_decay(t.end * 0.6931471805599453f);
      }
      __syncwarp();
      if (lane == 0) arrive(&b_tab[odd]);
    }
    if (lane == 0) {
#pragma unroll
      for (int hh = 0; hh < HPC; ++hh) f.tabs[(2 + odd) * HPC * kQ + hh] = total[hh];  // past both buffers
    }
    __syncwarp();
  } else {
    const int q4 = warp & 3, cg = warp >> 2;
    const int row = 32 * q4 + lane;
    const uint32_t tq = tmem + ((uint32_t)(32 * q4) << 16);
    const int hr = HPC == 2 ? row >> 6 : 0, p = PB == 64 ? row & 63 : row;
    float st[kSC];
#pragma unroll
    for (int i = 0; i < kSC; ++i) st[i] = 0.f;
    bool ok = true;
    if (kept != nullptr && s.first) {
      const size_t at = ((size_t)s.b * a.Hv + h0) * a.dv * DK;
      for (int e = 4 * tid; e < HPC * a.dv * DK; e += 4 * 32 * kWorkers)
        *reinterpret_cast<float4*>(kept + at + e) = *reinterpret_cast<const float4*>(init + at + e);
    }
    SsmDecay decay = {1.f, 0.f};  // of the chunk whose sum comes next
    auto update = [&](int c) {    // S after chunk c
      if (!(ok = wait(b_d, (uint32_t)(c & 1), 1))) return;
      tc::fence_after();
      float ds[kSC];
      tmem_load<kSC>(tq + kSum + kSC * cg, ds);
#pragma unroll
      for (int i = 0; i < kSC; i += 2) {
        const float2 v = make_float2(st[i], st[i + 1]);
        const float2 r = fma2(make_float2(decay.keep, decay.keep), v,
                              fma2(make_float2(decay.more, decay.more), v, make_float2(ds[i], ds[i + 1])));
        st[i] = r.x;
        st[i + 1] = r.y;
      }
    };
    for (int c = 0; c < nc; ++c) {
      const float* w = f.tabs + ((c & 1) * HPC + hr) * kQ;
      const unsigned char* xt = f.sm + (c % kSegStages) * C::kStage + C::kOffX;
      ok = wait(&b_st[c % kSegStages], (uint32_t)((c / kSegStages) & 1), 2) &&
           wait(&b_tab[c & 1], (uint32_t)((c >> 1) & 1), 1);
      if (!ok) break;
      if (32 * q4 < C::kRows) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          XwTiles xw;
          load_xw(xw, xt, w, lane, 32 * q4, 64 * hf + 16 * cg);
          split_xw(xw, tq + xw_col(c, hf) + 8 * cg);
        }
      }
      if (c > 0) update(c - 1);
      if (!ok) break;
      decay = f.lend[(c & 1) * HPC + hr];
      tmem_st_wait();
      tc::fence_before();
      __syncwarp();
      if (lane == 0) arrive(&w_a[c & 1]);
    }
    if (ok) update(nc - 1);
    if (ok && row < C::kRows && p < a.dv) {
      float4* dst = reinterpret_cast<float4*>(seg_state + seg_at<C>(s.slot, nhb, h0 / HPC, tid));
#pragma unroll
      for (int u = 0; u < kSC / 4; ++u)
        dst[u * 32 * kWorkers] = make_float4(st[4 * u], st[4 * u + 1], st[4 * u + 2], st[4 * u + 3]);
    }
  }
  if (gave_up != 0 && lane == 0) {
    *f.abort_flag = 1;
    atomicOr(err, gave_up);
  }
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  if (!*f.abort_flag && tid < HPC)
    seg_decay[(size_t)s.slot * a.Hv + h0 + tid] = f.tabs[2 * HPC * kQ + tid] + f.tabs[3 * HPC * kQ + tid];
  if (*f.abort_flag) {
    if (tid == 0) {
      for (int i = 0; i < 1 + kSegStages; ++i)
        for (uint32_t par = 0; par < 2; ++par) (void)tc::mbar_wait(&f.bars[i], par, 1u << 14);
    }
    __syncthreads();
  }
  if (warp == kAllocWarp) {
    __syncwarp();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

template <int DK, int PB, int HPC>
cudaError_t launch(const Maps& m, const SsmArgs& a, const Segs& g, float* seg_state, float* seg_decay,
                   const float* init, float* kept, float* fin, int* err, int phase, cudaStream_t st) {
  using C = Cfg<DK, PB, HPC>;
  const unsigned grid = (unsigned)(a.Hv / HPC) * (unsigned)g.slots;
  if (phase == 0) {
    const cudaError_t e = set_smem_limit_once<gdn_ssm_segment_kernel<DK, PB, HPC>>(C::kSmemBytes);
    if (e != cudaSuccess) return e;
    gdn_ssm_segment_kernel<DK, PB, HPC>
        <<<grid, kThreads, C::kSmemBytes, st>>>(m.x, m.b, a, g, seg_state, seg_decay, init, kept, err);
    return cudaGetLastError();
  }
  cudaError_t e = set_smem_limit_once<gdn_ssm_chunk_kernel<DK, PB, HPC>>(C::kSmemBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = g.len != 0 ? 1 : 0;  // behind the passes before it in the same call
  e = cudaLaunchKernelEx(&cfg, gdn_ssm_chunk_kernel<DK, PB, HPC>, m.x, m.b, m.c, m.z, m.out, a, g,
                         (const float*)seg_state, (const float*)seg_decay, init, (const float*)kept, fin, err);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

template <int DK>
cudaError_t launch_dk(const Maps& m, const SsmArgs& a, const Segs& g, float* seg_state, float* seg_decay,
                      const float* init, float* kept, float* fin, int* err, int hpc, int phase, cudaStream_t st) {
  if (a.dv == 128) return launch<DK, 128, 1>(m, a, g, seg_state, seg_decay, init, kept, fin, err, phase, st);
  if (hpc == 2) return launch<DK, 64, 2>(m, a, g, seg_state, seg_decay, init, kept, fin, err, phase, st);
  return launch<DK, 64, 1>(m, a, g, seg_state, seg_decay, init, kept, fin, err, phase, st);
}

}  // namespace ssm
}  // namespace gdn
