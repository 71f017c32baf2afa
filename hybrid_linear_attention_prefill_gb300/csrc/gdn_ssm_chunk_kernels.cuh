// The kernels of the chunked selective scan (gdn_ssm_chunk.cuh has the mathematics); one translation
// unit per state width instantiates them.
#pragma once

#include "gdn_ssm_chunk.cuh"

namespace gdn {
namespace ssm {

constexpr int kBars = 14;

// What both kernels set up: shared memory from a 1024-byte boundary, TMEM, barriers.
struct Frame {
  unsigned char* sm;
  uint32_t sb;  // shared-window address of sm
  uint64_t* bars;
  uint32_t* tmem_slot;
  volatile int* abort_flag;
  SsmDecay* lend;  // [2 buffers][heads]: e^{L_last}
  float* tabs;
};
template <class C>
__device__ __forceinline__ Frame make_frame(unsigned char* raw) {
  const uint32_t r = smem_u32(raw), pad = ((r + 1023u) & ~1023u) - r;
  Frame f;
  f.sm = raw + pad;
  f.sb = r + pad;
  f.bars = reinterpret_cast<uint64_t*>(f.sm + C::kOffBar);
  f.tmem_slot = reinterpret_cast<uint32_t*>(f.bars + kBars);
  f.abort_flag = reinterpret_cast<volatile int*>(f.tmem_slot + 1);
  f.lend = reinterpret_cast<SsmDecay*>(f.tmem_slot + 2);
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

// Outputs (and the final state of a sequence's last segment) of one segment and head block.
// grid: segments x head blocks, the head blocks of a segment side by side (they read the same B and C).
template <int DK, int PB, int HPC>
__global__ void __launch_bounds__(kThreads, 1)
gdn_ssm_chunk_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_b,
                     const __grid_constant__ CUtensorMap tm_c, const __grid_constant__ CUtensorMap tm_z,
                     const __grid_constant__ CUtensorMap tm_o, const SsmArgs a, const Segs g,
                     const float* seg_state, const float* init, float* fin, int* __restrict__ err) {
  using C = Cfg<DK, PB, HPC>;
  extern __shared__ unsigned char smem_raw[];
  const Frame f = make_frame<C>(smem_raw);
  // Completed by the MMAs, once a chunk each: scores, (w x)^T B of half 0 and C S^T, (w x)^T B of half 1, y.  By
  // copies: the two stages, C, the gate's tile.  By the worker warps: the first operands of a chunk (the state,
  // w x), the second (M, y, w x), the gate read, y read, the outputs out of the x tile.  By the table warp: a
  // chunk's tables, its stage loaded.
  uint64_t *b_sc = f.bars, *b_in = f.bars + 1, *b_d1 = f.bars + 2, *b_y = f.bars + 3, *b_st = f.bars + 4,
           *b_c = f.bars + 6, *b_z = f.bars + 7, *w_a = f.bars + 8, *w_b = f.bars + 9, *w_z = f.bars + 10,
           *w_y = f.bars + 11, *w_s = f.bars + 12, *b_tab = f.bars + 13;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp == kIssueWarp) {
    tc::tmem_alloc(f.tmem_slot, kTmemCols);
    tc::tmem_relinquish();
    if (lane == 0 && g.T > 0) {
      tc::prefetch_tensormap(&tm_x);
      tc::prefetch_tensormap(&tm_b);
      tc::prefetch_tensormap(&tm_c);
      if (a.z != nullptr) tc::prefetch_tensormap(&tm_z);
    }
  }
  if (tid == 0) {
    for (int i = 0; i < kBars; ++i) tc::mbar_init(&f.bars[i], i >= 8 && i < 13 ? kWorkers : 1);
    tc::fence_mbar_init();
    *f.abort_flag = 0;
  }
  asm volatile("griddepcontrol.wait;\n" ::: "memory");  // the segments' start states

  const int nhb = a.Hv / HPC, seg = blockIdx.x / nhb;
  const int h0 = (blockIdx.x - seg * nhb) * HPC;
  const int hk = h0 / (a.Hv / a.Hk);
  Seg s;
  const bool live = find_seg(g, seg, s);
  if (!live) s.t0 = s.t1 = 0, s.b = 0, s.bos = 0, s.slot = 0, s.first = s.last = false;
  const int ntok = s.t1 - s.t0, nc = (ntok + kQ - 1) / kQ;
  const long long tok0 = s.bos + s.t0;
  if (g.cu != nullptr && h0 == 0 && live && s.first && tid == 0) {
    const int lo = g.cu[s.b], hi = g.cu[s.b + 1];
    if (lo < 0 || hi < lo || hi > g.T || (s.b == 0 && lo != 0) || (s.b == g.B - 1 && hi != g.T)) atomicOr(err, 8);
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *f.tmem_slot;
  auto wait1 = [&](uint64_t* bar, uint32_t par, int bit) { return wait_for(bar, par, f.abort_flag, err, bit); };
  auto wait = [&](uint64_t* bar, uint32_t par, int bit) {  // a whole warp
    const bool done = wait1(bar, par, bit);
    __syncwarp();
    return done;
  };

  if (warp == kIssueWarp) {
    // ================= copies and MMAs: one thread =================
    auto load = [&](int c) {
      load_stage<DK, PB, C>(f, c & 1, &tm_b, &tm_x, hk, h0, a.dv, (int)(tok0 + (long long)c * kQ), &b_st[c & 1]);
    };
    auto load_c = [&](int c) {
      const int t = (int)(tok0 + (long long)c * kQ);
      tc::mbar_arrive_expect_tx(b_c, C::kNB * 16384);
#pragma unroll
      for (int i = 0; i < C::kNB; ++i) tc::tma_load_2d(f.sm + C::kOffC + i * 16384, &tm_c, hk * DK + 64 * i, t, b_c);
    };
    auto load_z = [&](int c) {
      const int t = (int)(tok0 + (long long)c * kQ);
      tc::mbar_arrive_expect_tx(b_z, C::kXB * 16384);
#pragma unroll
      for (int i = 0; i < C::kXB; ++i)
        tc::tma_load_2d(f.sm + C::kOffS + i * 16384, &tm_z, PB == 64 ? (h0 + i) * a.dv : h0 * a.dv + 64 * i, t, b_z);
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
      load(0);
      load_c(0);
      if (nc > 1) load(1);
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
        if (c + 1 < nc || a.z != nullptr) {
          if (!(ok = wait1(b_in, par, 1))) break;
          if (a.z != nullptr) load_z(c);  // over the state operand
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
      // The tables of chunk c - 2 were read up to its second operands.  Every phase is waited for in turn: a
      // parity names the last phase that ended, whichever that is.
      if (c > 1 && !wait(w_b, (uint32_t)(c & 1), 1)) break;
#pragma unroll
      for (int hh = 0; hh < HPC; ++hh) {
        float d[4];
        to_steps(a, ntok - c * kQ, bias[hh], lane, raw[hh], d);
        if (c + 1 < nc) load_dt(a, tok0 + (long long)(c + 1) * kQ, ntok - (c + 1) * kQ, h0 + hh, lane, raw[hh]);
        const float end = make_tables<false>(f.tabs + (c & 1) * (C::kTab / 4) + hh * 3 * kQ, d, a_log2[hh], lane);
        if (lane == 0) f.lend[(c & 1) * HPC + hh] = ssm_decay(end * 0.6931471805599453f);
      }
      if (!wait(&b_st[c & 1], (uint32_t)((c >> 1) & 1), 2)) break;
      if (lane == 0) arrive(b_tab);
      if (lane == 0) {  // into L2, where their places in shared memory are free only late: this chunk's gate, the next x and B
        const int t = (int)(tok0 + (long long)c * kQ);
#pragma unroll
        for (int i = 0; i < C::kXB; ++i) {
          const int col = PB == 64 ? (h0 + i) * a.dv : h0 * a.dv + 64 * i;
          if (a.z != nullptr) tma_prefetch_l2_2d(&tm_z, col, t);
          if (c > 0 && c + 1 < nc) tma_prefetch_l2_2d(&tm_x, col, t + kQ);
        }
        if (c > 0 && c + 1 < nc)
#pragma unroll
          for (int i = 0; i < C::kNB; ++i) tma_prefetch_l2_2d(&tm_b, hk * DK + 64 * i, t + kQ);
      }
      __syncwarp();
    }
  } else {
    // ================= workers =================
    const int q4 = warp & 3, cg = warp >> 2;
    const int row = 32 * q4 + lane;  // state row, or token of the chunk
    const uint32_t tq = tmem + ((uint32_t)(32 * q4) << 16);
    // this thread's state: row (head, p), columns kSC cg ..
    const int hr = HPC == 2 ? row >> 6 : 0, p = PB == 64 ? row & 63 : row;
    const bool my_row = live && row < C::kRows && p < a.dv;
    float st[C::kSC];
    {
      const float* src = g.len != 0 ? seg_state + (size_t)s.slot * a.Hv * a.dv * DK
                                    : init != nullptr ? init + (size_t)s.b * a.Hv * a.dv * DK : nullptr;
#pragma unroll
      for (int i = 0; i < C::kSC; i += 4) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (my_row && src != nullptr)
          v = *reinterpret_cast<const float4*>(src + ((size_t)(h0 + hr) * a.dv + p) * DK + C::kSC * cg + i);
        st[i] = v.x; st[i + 1] = v.y; st[i + 2] = v.z; st[i + 3] = v.w;
      }
    }
    // this warp's outputs: tokens 32 q4 .. + 31, columns kYC cg .., worked on by rows in the warp's own part of the
    // x tile and stored from there in memory order (kP 16-byte pieces a token)
    constexpr int kP = C::kYC / 8;
    const int yc = C::kYC * cg;
    const int yh = HPC == 2 ? yc >> 6 : 0, yp = PB == 64 ? yc & 63 : yc;
    const bool my_cols = yp < a.dv;
    const float skip = a.D != nullptr && my_cols ? a.D[h0 + yh] : 0.f;
    const int mt = 32 * q4 + lane / kP, mp = lane % kP;  // memory order: token mt + (32 / kP) i, piece mp
    const int quad = 2 + 4 * (yc >> 6) + q4;  // named barrier of the warps that share 32 tokens of a 64-wide block
    const uint32_t yoff = (uint32_t)(yc >> 6) * 16384, ych = (uint32_t)(yc & 63) >> 3;
    const bool gate = a.z != nullptr;

    bool ok = true;
    // The first operands of chunk c: the state, and w x of its first 64 tokens.
    auto first_operands = [&](int c) {
      unsigned char* stage = f.sm + (c & 1) * C::kStage;
      const int n = min(kQ, ntok - c * kQ);
      if (!wait(b_tab, (uint32_t)(c & 1), 1)) return false;
      if (n < kQ) {  // rows of the sequence after this one: zeros, so that no value of theirs meets a zero weight
        const int rows = kQ - n;
        for (int e = tid; e < rows * 8 * (C::kNB + C::kXB); e += 32 * kWorkers)
          *reinterpret_cast<uint4*>(stage + (e / (rows * 8)) * 16384 + (n * 8 + e % (rows * 8)) * 16) =
              make_uint4(0, 0, 0, 0);
        asm volatile("bar.sync 1, %0;\n" ::"n"(32 * kWorkers) : "memory");
      }
      if (gate && c > 0 && !wait(w_z, (uint32_t)((c - 1) & 1), 1)) return false;  // every warp has read the gate there
      if (row < C::kRows) {
#pragma unroll
        for (int i = 0; i < C::kSC; i += 8) {
          const int col = C::kSC * cg + i;
          *reinterpret_cast<uint4*>(f.sm + C::kOffS + (col >> 6) * (C::kRows * 128) +
                                    tc::sw128((uint32_t)row, (uint32_t)(col & 63) >> 3)) =
              make_uint4(pack_bf16(st[i], st[i + 1]), pack_bf16(st[i + 2], st[i + 3]), pack_bf16(st[i + 4], st[i + 5]),
                         pack_bf16(st[i + 6], st[i + 7]));
        }
      }
      const float* tab = f.tabs + (c & 1) * (C::kTab / 4);
      if (32 * q4 < C::kRows)
        split_xw(stage + C::kOffX, tab + hr * 3 * kQ + 2 * kQ, 32 * q4, 16 * cg, tq + kColXw + 8 * cg);
      tmem_st_wait();
      tc::fence_proxy_async();
      tc::fence_before();
      __syncwarp();
      if (lane == 0) arrive(w_a);
      return true;
    };
    if (nc > 0) ok = first_operands(0);
    for (int c = 0; ok && c < nc; ++c) {
      const uint32_t par = (uint32_t)(c & 1);
      unsigned char* xt = f.sm + (c & 1) * C::kStage + C::kOffX;
      unsigned char* yt = xt + yoff;
      const float* tab = f.tabs + (c & 1) * (C::kTab / 4);
      const int n = min(kQ, ntok - c * kQ);

      // ---- M from the scores, in their place: eight columns a head of each 16 ------------------------
      if (!(ok = wait(b_sc, par, 1))) break;
      tc::fence_after();
#pragma unroll
      for (int j0 = 0; j0 < 32; j0 += 16) {
        const uint32_t col = tq + kColSc + 32 * cg + j0;
        uint32_t m[8];
        if (cg <= q4) {
          float sc[16];
          tc::tmem_ld16(col, sc);
#pragma unroll
          for (int hh = 0; hh < HPC; ++hh) {
            const float* th = tab + hh * 3 * kQ;
            const float li = th[row];
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
              const float4 k4 = *reinterpret_cast<const float4*>(th + kQ + 32 * cg + j0 + j);
              const float2 minus = make_float2(-1.f, -1.f), l2 = make_float2(li, li);
              const float2 e0 = fma2(make_float2(k4.x, k4.y), minus, l2), e1 = fma2(make_float2(k4.z, k4.w), minus, l2);
              float2 u = mul2(make_float2(sc[j], sc[j + 1]), make_float2(ex2_approx(e0.x), ex2_approx(e0.y)));
              float2 v = mul2(make_float2(sc[j + 2], sc[j + 3]), make_float2(ex2_approx(e1.x), ex2_approx(e1.y)));
              if (cg == q4) {
                u.x = j0 + j <= lane ? u.x : 0.f;
                u.y = j0 + j + 1 <= lane ? u.y : 0.f;
                v.x = j0 + j + 2 <= lane ? v.x : 0.f;
                v.y = j0 + j + 3 <= lane ? v.y : 0.f;
              }
              m[j / 2] = pack_bf16(u.x, u.y);
              m[j / 2 + 1] = pack_bf16(v.x, v.y);
            }
            tmem_st8_nowait(col + 8 * hh, m);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) m[j] = 0u;
#pragma unroll
          for (int hh = 0; hh < HPC; ++hh) tmem_st8_nowait(col + 8 * hh, m);
        }
      }
      if (c > 0) {  // the chunk before's outputs have left its x tile
        bulk_wait_read();
        __syncwarp();
        if (lane == 0) arrive(w_s);
      }
      // ---- y = e^{L_i} (C S^T), in place; w x of the other 64 tokens ----------------------------------
      if (!(ok = wait(b_in, par, 1))) break;  // and (w x)^T B of the first 64 before it
      tc::fence_after();
      {
        float y[C::kYC];
        tmem_load<C::kYC>(tq + kColY + yc, y);
        const float e = exp2f(tab[yh * 3 * kQ + row]);
        uint32_t u[C::kYC];
#pragma unroll
        for (int i = 0; i < C::kYC; i += 2) {
          const float2 v = mul2(make_float2(y[i], y[i + 1]), make_float2(e, e));
          u[i] = __float_as_uint(v.x);
          u[i + 1] = __float_as_uint(v.y);
        }
#pragma unroll
        for (int i = 0; i < C::kYC; i += 16)
          tmem_st16_nowait(tq + kColY + yc + i, reinterpret_cast<const uint32_t(&)[16]>(u[i]));
      }
      if (32 * q4 < C::kRows) split_xw(xt, tab + hr * 3 * kQ + 2 * kQ, 32 * q4, 64 + 16 * cg, tq + kColXw + 8 * cg);
      tmem_st_wait();
      tc::fence_before();
      __syncwarp();
      if (lane == 0) arrive(w_b);

      // ---- the gate -------------------------------------------------------------------------------------
      // Of this thread's row of the gate, half goes through silu while M x runs; the rest waits as it is (all of
      // it would not fit the registers).
      uint4 zr[kP];
      float2 gv[2 * kP];
      auto gates = [&](int i, int u) {
        const uint32_t w = u == 0 ? zr[i].x : u == 1 ? zr[i].y : u == 2 ? zr[i].z : zr[i].w;
        return silu2(make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)));
      };
      if (gate) {
        if (!(ok = wait(b_z, par, 2))) break;
        const unsigned char* zt = f.sm + C::kOffS + yoff;
#pragma unroll
        for (int i = 0; i < kP; ++i) zr[i] = *reinterpret_cast<const uint4*>(zt + tc::sw128((uint32_t)row, ych + i));
        __syncwarp();
        if (lane == 0) arrive(w_z);
#pragma unroll
        for (int i = 0; i < kP / 2; ++i)
#pragma unroll
          for (int u = 0; u < 4; ++u) gv[4 * i + u] = gates(i, u);
      }
      // ---- S = e^{L_last} S + the chunk's sum ---------------------------------------------------------
      if (!(ok = wait(b_d1, par, 1))) break;
      tc::fence_after();
      {
        float ds[C::kSC];
        tmem_load<C::kSC>(tq + kColDs + C::kSC * cg, ds);
        const SsmDecay decay = f.lend[(c & 1) * HPC + hr];
#pragma unroll
        for (int i = 0; i < C::kSC; i += 2) {
          const float2 v = make_float2(st[i], st[i + 1]);
          const float2 r = fma2(make_float2(decay.keep, decay.keep), v,
                                fma2(make_float2(decay.more, decay.more), v, make_float2(ds[i], ds[i + 1])));
          st[i] = r.x;
          st[i + 1] = r.y;
        }
      }
      if (c + 1 < nc && !(ok = first_operands(c + 1))) break;
      // ---- outputs, by way of the warp's own part of the x tile -----------------------------------------
      if (!(ok = wait(b_y, par, 1))) break;
      tc::fence_after();
      {
        for (int i0 = 0; i0 < kP; i0 += 2) {  // sixteen columns of this thread's own row at a time
          float y[16];
          tc::tmem_ld16(tq + kColY + yc + 8 * i0, y);
          if (i0 + 2 == kP) {
            tc::fence_before();
            __syncwarp();
            if (lane == 0) arrive(w_y);
          }
          uint4 x[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) x[i] = *reinterpret_cast<const uint4*>(yt + tc::sw128((uint32_t)row, ych + i0 + i));
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t x4[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
            float2 v[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              v[u] = fma2(make_float2(__uint_as_float(x4[u] << 16), __uint_as_float(x4[u] & 0xffff0000u)),
                          make_float2(skip, skip), make_float2(y[8 * i + 2 * u], y[8 * i + 2 * u + 1]));
              if (gate) v[u] = mul2(v[u], i0 + i < kP / 2 ? gv[4 * ((i0 + i) % (kP / 2)) + u] : gates(i0 + i, u));
            }
            *reinterpret_cast<uint4*>(yt + tc::sw128((uint32_t)row, ych + i0 + i)) = make_uint4(
                pack_bf16(v[0].x, v[0].y), pack_bf16(v[1].x, v[1].y), pack_bf16(v[2].x, v[2].y), pack_bf16(v[3].x, v[3].y));
          }
        }
        if (a.dv >= 64 && 32 * q4 + 32 <= n) {  // 32 whole tokens of 64 columns: one copy by the first of their warps
          tc::fence_proxy_async();
          asm volatile("bar.sync %0, %1;\n" ::"r"(quad), "n"(32 * (64 / C::kYC)) : "memory");
          if ((yc & 63) == 0 && lane == 0) {
            tma_store_2d(&tm_o, smem_u32(yt) + 32 * q4 * 128, (h0 + yh) * a.dv + yp, (int)(tok0 + (long long)c * kQ) + 32 * q4);
            bulk_commit();
          }
          __syncwarp();
        } else {
          __syncwarp();
          if (my_cols) {
            __nv_bfloat16* o = a.out + ((size_t)(tok0 + (long long)c * kQ) * a.Hv + h0 + yh) * a.dv + yp + 8 * mp;
#pragma unroll
            for (int i = 0; i < kP; ++i) {
              const int t = mt + (32 / kP) * i;
              if (t < n)
                *reinterpret_cast<uint4*>(o + (size_t)t * a.Hv * a.dv) =
                    *reinterpret_cast<const uint4*>(yt + tc::sw128((uint32_t)t, ych + mp));
            }
          }
          tc::fence_proxy_async();
        }
      }
    }
    bulk_wait_read();
    if (!ok) {  // another warp may have passed the wait that this one gave up, and stand at a barrier between warps
      asm volatile("bar.arrive 1, %0;\n" ::"n"(32 * kWorkers) : "memory");
      asm volatile("bar.arrive %0, %1;\n" ::"r"(quad), "n"(32 * (64 / C::kYC)) : "memory");
    }
    if (ok && fin != nullptr && s.last && my_row) {
      float* dst = fin + (((size_t)s.b * a.Hv + h0 + hr) * a.dv + p) * DK + C::kSC * cg;
#pragma unroll
      for (int i = 0; i < C::kSC; i += 4)
        *reinterpret_cast<float4*>(dst + i) = make_float4(st[i], st[i + 1], st[i + 2], st[i + 3]);
    }
  }
  tc::fence_before();
  __syncthreads();
  if (*f.abort_flag && warp == kIssueWarp && lane == 0) {  // let what is in flight land, bounded again
    for (int i = 0; i < 8; ++i)
      for (uint32_t par = 0; par < 2; ++par) (void)tc::mbar_wait(&f.bars[i], par, 1u << 14);
  }
  __syncwarp();
  if (warp == kIssueWarp) tc::tmem_dealloc(tmem, kTmemCols);
}

// The sums of the segments before a sequence's last (from a zero state) and their decays in log2.
// grid: segments x head blocks.
template <int DK, int PB, int HPC>
__global__ void __launch_bounds__(kThreads, 1)
gdn_ssm_segment_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_b,
                       const SsmArgs a, const Segs g, float* __restrict__ seg_state, float* __restrict__ seg_decay,
                       int* __restrict__ err) {
  using C = Cfg<DK, PB, HPC>;
  extern __shared__ unsigned char smem_raw[];
  const Frame f = make_frame<C>(smem_raw);
  uint64_t *b_d = f.bars, *b_st = f.bars + 1, *w_a = f.bars + 8, *b_tab = f.bars + 13;
  const int nhb = a.Hv / HPC, seg = blockIdx.x / nhb;
  Seg s;
  if (!find_seg(g, seg, s) || s.last) return;  // a last segment's sum is nobody's start
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp == kIssueWarp) {
    tc::tmem_alloc(f.tmem_slot, kTmemCols);
    tc::tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < kBars; ++i) tc::mbar_init(&f.bars[i], i == 8 ? kWorkers : 1);
    tc::fence_mbar_init();
    *f.abort_flag = 0;
  }
  const int h0 = (blockIdx.x - seg * nhb) * HPC;
  const int hk = h0 / (a.Hv / a.Hk);
  const int nc = (s.t1 - s.t0) / kQ;  // whole chunks: only a last segment is ragged
  const long long tok0 = s.bos + s.t0;
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *f.tmem_slot;
  auto wait1 = [&](uint64_t* bar, uint32_t par, int bit) { return wait_for(bar, par, f.abort_flag, err, bit); };
  auto wait = [&](uint64_t* bar, uint32_t par, int bit) {  // a whole warp
    const bool done = wait1(bar, par, bit);
    __syncwarp();
    return done;
  };
  // TMEM: w x of a chunk (two halves of 96 columns) in two buffers, the sum between them
  constexpr uint32_t kSum = 288;
  auto xw_col = [](int c, int hf) { return (uint32_t)((c & 1) ? (hf ? 416 : 192) : (hf ? 96 : 0)); };

  if (warp == kIssueWarp) {
    auto load = [&](int c) {
      load_stage<DK, PB, C>(f, c & 1, &tm_b, &tm_x, hk, h0, a.dv, (int)(tok0 + (long long)c * kQ), &b_st[c & 1]);
    };
    if (lane == 0) {
      load(0);
      if (nc > 1) load(1);
      for (int c = 0; c < nc; ++c) {
        if (!wait1(w_a, (uint32_t)(c & 1), 1)) break;  // w x of chunk c written, the sum of c - 1 read
        tc::fence_after();
        if (c > 0 && c + 1 < nc) load(c + 1);
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
          issue_state<DK>(tmem + kSum, tmem + xw_col(c, hf), f.sb + (c & 1) * C::kStage + C::kOffB, hf, hf == 0);
        tc::commit(b_d);
      }
    }
    __syncwarp();
  } else if (warp == kTableWarp) {
    float a_log2[HPC], bias[HPC], total[HPC];
    uint32_t raw[HPC][4];
#pragma unroll
    for (int hh = 0; hh < HPC; ++hh) {
      a_log2[hh] = a.A[h0 + hh] * 1.4426950408889634f;
      bias[hh] = ssm_bias(a, h0 + hh);
      total[hh] = 0.f;
      load_dt(a, tok0, kQ, h0 + hh, lane, raw[hh]);
    }
    for (int c = 0; c < nc; ++c) {
      if (c > 0 && !wait(w_a, (uint32_t)((c - 1) & 1), 1)) break;
#pragma unroll
      for (int hh = 0; hh < HPC; ++hh) {
        float d[4];
        to_steps(a, kQ, bias[hh], lane, raw[hh], d);
        if (c + 1 < nc) load_dt(a, tok0 + (long long)(c + 1) * kQ, kQ, h0 + hh, lane, raw[hh]);
        const float end = make_tables<true>(f.tabs + ((c & 1) * HPC + hh) * kQ, d, a_log2[hh], lane);
        total[hh] += end;
        if (lane == 0) f.lend[(c & 1) * HPC + hh] = ssm_decay(end * 0.6931471805599453f);
      }
      __syncwarp();
      if (lane == 0) arrive(b_tab);
    }
    if (lane == 0) {
#pragma unroll
      for (int hh = 0; hh < HPC; ++hh) seg_decay[(size_t)s.slot * a.Hv + h0 + hh] = total[hh];
    }
  } else {
    const int q4 = warp & 3, cg = warp >> 2;
    const int row = 32 * q4 + lane;
    const uint32_t tq = tmem + ((uint32_t)(32 * q4) << 16);
    const int hr = HPC == 2 ? row >> 6 : 0, p = PB == 64 ? row & 63 : row;
    float st[C::kSC];
#pragma unroll
    for (int i = 0; i < C::kSC; ++i) st[i] = 0.f;
    bool ok = true;
    SsmDecay decay = {1.f, 0.f};  // of the chunk whose sum comes next
    auto update = [&](int c) {    // S after chunk c
      if (!(ok = wait(b_d, (uint32_t)(c & 1), 1))) return;
      tc::fence_after();
      float ds[C::kSC];
      tmem_load<C::kSC>(tq + kSum + C::kSC * cg, ds);
#pragma unroll
      for (int i = 0; i < C::kSC; i += 2) {
        const float2 v = make_float2(st[i], st[i + 1]);
        const float2 r = fma2(make_float2(decay.keep, decay.keep), v,
                              fma2(make_float2(decay.more, decay.more), v, make_float2(ds[i], ds[i + 1])));
        st[i] = r.x;
        st[i + 1] = r.y;
      }
    };
    for (int c = 0; c < nc; ++c) {
      const float* w = f.tabs + ((c & 1) * HPC + hr) * kQ;
      const unsigned char* xt = f.sm + (c & 1) * C::kStage + C::kOffX;
      if (!(ok = wait(&b_st[c & 1], (uint32_t)((c >> 1) & 1), 2) && wait(b_tab, (uint32_t)(c & 1), 1))) break;
      if (32 * q4 < C::kRows) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) split_xw(xt, w, 32 * q4, 64 * hf + 16 * cg, tq + xw_col(c, hf) + 8 * cg);
      }
      if (c > 0) update(c - 1);
      if (!ok) break;
      decay = f.lend[(c & 1) * HPC + hr];
      tmem_st_wait();
      tc::fence_before();
      __syncwarp();
      if (lane == 0) arrive(w_a);
    }
    if (ok) update(nc - 1);
    if (ok && row < C::kRows && p < a.dv) {
      float* dst = seg_state + (((size_t)s.slot * a.Hv + h0 + hr) * a.dv + p) * DK + C::kSC * cg;
#pragma unroll
      for (int i = 0; i < C::kSC; i += 4)
        *reinterpret_cast<float4*>(dst + i) = make_float4(st[i], st[i + 1], st[i + 2], st[i + 3]);
    }
  }
  tc::fence_before();
  __syncthreads();
  if (*f.abort_flag && warp == kIssueWarp && lane == 0) {
    for (int i = 0; i < 3; ++i)
      for (uint32_t par = 0; par < 2; ++par) (void)tc::mbar_wait(&f.bars[i], par, 1u << 14);
  }
  __syncwarp();
  if (warp == kIssueWarp) tc::tmem_dealloc(tmem, kTmemCols);
}

template <int DK, int PB, int HPC>
cudaError_t launch(const Maps& m, const SsmArgs& a,
                   const Segs& g, float* seg_state, float* seg_decay, const float* init, float* fin, int* err,
                   int phase, cudaStream_t st) {
  using C = Cfg<DK, PB, HPC>;
  const unsigned grid = (unsigned)(a.Hv / HPC) * (unsigned)g.slots;
  if (phase == 0) {
    const cudaError_t e = set_smem_limit_once<gdn_ssm_segment_kernel<DK, PB, HPC>>(C::kSmemBytes);
    if (e != cudaSuccess) return e;
    gdn_ssm_segment_kernel<DK, PB, HPC><<<grid, kThreads, C::kSmemBytes, st>>>(m.x, m.b, a, g, seg_state, seg_decay, err);
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
  cfg.numAttrs = g.len != 0 ? 1 : 0;  // behind the combine kernel of the same call
  e = cudaLaunchKernelEx(&cfg, gdn_ssm_chunk_kernel<DK, PB, HPC>, m.x, m.b, m.c, m.z, m.out, a, g, (const float*)seg_state, init, fin,
                         err);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

template <int DK>
cudaError_t launch_dk(const Maps& m, const SsmArgs& a,
                      const Segs& g, float* seg_state, float* seg_decay, const float* init, float* fin, int* err,
                      int hpc, int phase, cudaStream_t st) {
  if (a.dv == 128) return launch<DK, 128, 1>(m, a, g, seg_state, seg_decay, init, fin, err, phase, st);
  if (hpc == 2) return launch<DK, 64, 2>(m, a, g, seg_state, seg_decay, init, fin, err, phase, st);
  return launch<DK, 64, 1>(m, a, g, seg_state, seg_decay, init, fin, err, phase, st);
}

}  // namespace ssm
}  // namespace gdn
