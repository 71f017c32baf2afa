// The kernels of the chunked selective scan (gdn_ssm_chunk.cuh has the mathematics); one translation
// unit per state width instantiates them.
#pragma once

#include "gdn_ssm_chunk.cuh"

namespace gdn {
namespace ssm {

// Outputs (and the final state of a sequence's last segment) of one segment and head block.
// grid: segments x head blocks, the head blocks of a segment side by side (they read the same B and C).
template <int DK, int PB, int HPC>
__global__ void __launch_bounds__(kThreads, 1)
gdn_ssm_chunk_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_b,
                     const __grid_constant__ CUtensorMap tm_c, const SsmArgs a, const Segs g,
                     const float* seg_state, const float* init, float* fin, int* __restrict__ err) {
  using C = Cfg<DK, PB, HPC>;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw_s = smem_u32(smem_raw);
  const uint32_t pad = ((raw_s + 1023u) & ~1023u) - raw_s;
  unsigned char* sm = smem_raw + pad;
  const uint32_t sb = raw_s + pad;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + C::kOffBar);
  // [0] scores, [1] C S^T, [2] state half 0, [3] y, [4] state half 1: each completes once a chunk;
  // [5], [6] stage loaded, [7] C loaded
  uint64_t *b_sc = bars, *b_in = bars + 1, *b_d0 = bars + 2, *b_y = bars + 3, *b_d1 = bars + 4, *b_st = bars + 5,
           *b_c = bars + 7;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  SsmDecay* lend = reinterpret_cast<SsmDecay*>(tmem_slot + 2);  // [2 buffers][HPC]: e^{L_last}
  float* tabs = reinterpret_cast<float*>(sm + C::kOffTab);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int q4 = warp & 3, cg = warp >> 2;
  const int row = 32 * q4 + lane;  // state row, or token of the chunk
  // single-warp jobs go to warps whose part of M is above the diagonal
  const bool issuer = warp == 12 && lane == 0;
  const bool loader = warp == 4 && lane == 0;
  const int tab_head = warp == 8 ? 0 : (HPC == 2 && warp == 13) ? 1 : -1;

  if (warp == 12) {
    tc::tmem_alloc(tmem_slot, kTmemCols);
    tc::tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < 8; ++i) tc::mbar_init(&bars[i], 1);
    tc::fence_mbar_init();
    *abort_flag = 0;
  }
  if (loader && g.T > 0) {
    tc::prefetch_tensormap(&tm_x);
    tc::prefetch_tensormap(&tm_b);
    tc::prefetch_tensormap(&tm_c);
  }
  asm volatile("griddepcontrol.wait;\n" ::: "memory");  // the segments' start states

  const int nhb = a.Hv / HPC, seg = blockIdx.x / nhb;
  const int h0 = (blockIdx.x - seg * nhb) * HPC;
  const int hk = h0 / (a.Hv / a.Hk);
  Seg s;
  const bool live = find_seg(g, seg, s);
  if (!live) s.t0 = s.t1 = 0, s.b = 0, s.bos = 0, s.slot = 0, s.first = s.last = false;
  const int nc = (s.t1 - s.t0 + kQ - 1) / kQ;
  const long long tok0 = s.bos + s.t0;
  if (g.cu != nullptr && h0 == 0 && live && s.first && tid == 0) {
    const int lo = g.cu[s.b], hi = g.cu[s.b + 1];
    if (lo < 0 || hi < lo || hi > g.T || (s.b == 0 && lo != 0) || (s.b == g.B - 1 && hi != g.T)) atomicOr(err, 8);
  }

  // this thread's state: row (head, p), columns kSC cg .. ; the head's row of a 64-row block is p
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

  auto load_stage = [&](int c) {  // B and x of chunk c
    unsigned char* dst = sm + (c & 1) * C::kStage;
    uint64_t* bar = &b_st[c & 1];
    const int t = (int)(tok0 + (long long)c * kQ);
    tc::mbar_arrive_expect_tx(bar, C::kStage);
#pragma unroll
    for (int i = 0; i < C::kNB; ++i) tc::tma_load_2d(dst + C::kOffB + i * 16384, &tm_b, hk * DK + 64 * i, t, bar);
#pragma unroll
    for (int i = 0; i < C::kXB; ++i)
      tc::tma_load_2d(dst + C::kOffX + i * 16384, &tm_x, PB == 64 ? (h0 + i) * a.dv : h0 * a.dv + 64 * i, t, bar);
  };
  auto load_c = [&](int c) {
    const int t = (int)(tok0 + (long long)c * kQ);
    tc::mbar_arrive_expect_tx(b_c, C::kNB * 16384);
#pragma unroll
    for (int i = 0; i < C::kNB; ++i) tc::tma_load_2d(sm + C::kOffC + i * 16384, &tm_c, hk * DK + 64 * i, t, b_c);
  };
  auto wait = [&](uint64_t* bar, uint32_t par, int bit) {
    if (!tc::mbar_wait(bar, par, kMaxPolls)) {
      *abort_flag = 1;
      atomicOr(err, bit);
    }
  };
  // scores of chunk c: C_i . B_j over the chunk's tokens, once both tiles are in
  auto issue_scores = [&](int c) {
    wait(&b_st[c & 1], (uint32_t)((c >> 1) & 1), 2);
    wait(b_c, (uint32_t)(c & 1), 2);
    constexpr uint32_t kId = tc::idesc_bf16(128, 128, 0, 0);
    const uint64_t ad = tc::sdesc(sb + C::kOffC, 16, 1024, tc::kSw128);
    const uint64_t bd = tc::sdesc(sb + (c & 1) * C::kStage + C::kOffB, 16, 1024, tc::kSw128);
#pragma unroll
    for (int ks = 0; ks < DK / 16; ++ks) {
      const uint64_t off = (uint64_t)(((ks >> 2) * 16384 + (ks & 3) * 32) >> 4);
      tc::mma_bf16(*tmem_slot + kColSc, ad + off, bd + off, kId, ks > 0);
    }
    tc::commit(b_sc);
  };

  // the steps of the next chunk whose tables this warp will make
  float d[4] = {0.f, 0.f, 0.f, 0.f};
  const float a_log2 = tab_head >= 0 ? a.A[h0 + tab_head] * 1.4426950408889634f : 0.f;
  auto tables = [&](int c) {  // from d; then chunk c + 1's steps into d
    float* tab = tabs + (c & 1) * (C::kTab / 4) + tab_head * 3 * kQ;
    const float end = make_tables<false>(tab, d, a_log2, lane);
    if (lane == 0) lend[(c & 1) * HPC + tab_head] = ssm_decay(end * 0.6931471805599453f);
    if (c + 1 < nc) load_steps(a, tok0 + (long long)(c + 1) * kQ, s.t1 - s.t0 - (c + 1) * kQ, h0 + tab_head, lane, d);
  };

  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tq = tmem + ((uint32_t)(32 * q4) << 16);
  if (nc > 0) {
    if (loader) {
      load_stage(0);
      load_c(0);
      if (nc > 1) load_stage(1);
    }
    if (tab_head >= 0) {
      load_steps(a, tok0, s.t1 - s.t0, h0 + tab_head, lane, d);
      tables(0);
    }
    if (issuer) issue_scores(0);
    __syncthreads();  // the first tables
  }

  // this thread's output columns
  const int yc = C::kYC * cg;
  const int yh = HPC == 2 ? yc >> 6 : 0, yp = PB == 64 ? yc & 63 : yc;
  const bool my_cols = yp < a.dv;
  const float skip = a.D != nullptr && my_cols ? a.D[h0 + yh] : 0.f;

  // the outputs of chunk c, staged over its x tile, to memory: 16 bytes a thread, rows in order
  auto copy_out = [&](int c) {
    const unsigned char* xt = sm + (c & 1) * C::kStage + C::kOffX;
    const int n = min(kQ, s.t1 - s.t0 - c * kQ);
    const int per_head = a.dv >> 3, sh = a.dv == 128 ? 4 : a.dv == 64 ? 3 : 2;  // 16-byte pieces
    __nv_bfloat16* o = a.out + ((size_t)(tok0 + (long long)c * kQ) * a.Hv + h0) * a.dv;
    for (int e = tid; e < n * per_head * HPC; e += kThreads) {
      const int piece = e & (per_head - 1), th = e >> sh;
      const int hh = HPC == 2 ? th & 1 : 0, t = HPC == 2 ? th >> 1 : th;
      const int col = PB == 64 ? 64 * hh + 8 * piece : 8 * piece;
      *reinterpret_cast<uint4*>(o + ((size_t)t * a.Hv + hh) * a.dv + 8 * piece) =
          *reinterpret_cast<const uint4*>(xt + (col >> 6) * 16384 + tc::sw128((uint32_t)t, (uint32_t)(col & 63) >> 3));
    }
  };

  bool aborted = false;
  for (int c = 0; c < nc; ++c) {
    const uint32_t par = (uint32_t)(c & 1);
    unsigned char* stage = sm + (c & 1) * C::kStage;
    unsigned char* xt = stage + C::kOffX;
    const float* tab = tabs + (c & 1) * (C::kTab / 4);
    const int n = min(kQ, s.t1 - s.t0 - c * kQ);

    wait(&b_st[c & 1], (uint32_t)((c >> 1) & 1), 2);
    if (n < kQ) {  // rows of the sequence after this one: zeros, so that no value of theirs meets a zero weight
      const int rows = kQ - n;
      for (int e = tid; e < rows * 8 * (C::kNB + C::kXB); e += kThreads)
        *reinterpret_cast<uint4*>(stage + (e / (rows * 8)) * 16384 + (n * 8 + e % (rows * 8)) * 16) = make_uint4(0, 0, 0, 0);
      __syncthreads();
    }

    // ---- the state as an operand; w x of the first 64 tokens ------------------------------------
    if (row < C::kRows) {
#pragma unroll
      for (int i = 0; i < C::kSC; i += 8) {
        const int col = C::kSC * cg + i;
        *reinterpret_cast<uint4*>(sm + C::kOffS + (col >> 6) * (C::kRows * 128) +
                                  tc::sw128((uint32_t)row, (uint32_t)(col & 63) >> 3)) =
            make_uint4(pack_bf16(st[i], st[i + 1]), pack_bf16(st[i + 2], st[i + 3]), pack_bf16(st[i + 4], st[i + 5]),
                       pack_bf16(st[i + 6], st[i + 7]));
      }
    }
    if (32 * q4 < C::kRows) split_xw(xt, tab + hr * 3 * kQ + 2 * kQ, row, 16 * cg, tq + kColXw + 8 * cg);
    tmem_st_wait();
    tc::fence_proxy_async();
    tc::fence_before();
    __syncthreads();
    if (*abort_flag) { aborted = true; break; }
    if (issuer) {
      tc::fence_after();
      constexpr uint32_t kId = tc::idesc_bf16(128, C::kRows, 0, 0);
      const uint64_t ad = tc::sdesc(sb + C::kOffC, 16, 1024, tc::kSw128);
      const uint64_t bd = tc::sdesc(sb + C::kOffS, 16, 1024, tc::kSw128);
#pragma unroll
      for (int ks = 0; ks < DK / 16; ++ks)
        tc::mma_bf16(tmem + kColY, ad + (uint64_t)(((ks >> 2) * 16384 + (ks & 3) * 32) >> 4),
                     bd + (uint64_t)(((ks >> 2) * (C::kRows * 128) + (ks & 3) * 32) >> 4), kId, ks > 0);
      tc::commit(b_in);
      issue_state<DK>(tmem, tmem + kColXw, sb + (c & 1) * C::kStage + C::kOffB, 0, true);
      tc::commit(b_d0);
    }
    __syncwarp();

    // ---- meanwhile: the chunk before's outputs, the next tables, M ---------------------------------
    if (c > 0) copy_out(c - 1);
    if (tab_head >= 0 && c + 1 < nc) tables(c + 1);
    wait(b_sc, par, 1);
    tc::fence_after();
    {
      uint32_t m[HPC][16];
      if (cg <= q4) {
        float sc[32];
        tc::tmem_ld32(tq + kColSc + 32 * cg, sc);
#pragma unroll
        for (int hh = 0; hh < HPC; ++hh) {
          const float* th = tab + hh * 3 * kQ;
          const float li = th[row];
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            const float4 l4 = *reinterpret_cast<const float4*>(th + 32 * cg + j);
            const float4 s4 = *reinterpret_cast<const float4*>(th + kQ + 32 * cg + j);
            float v[4] = {sc[j] * s4.x * ex2(li - l4.x), sc[j + 1] * s4.y * ex2(li - l4.y),
                          sc[j + 2] * s4.z * ex2(li - l4.z), sc[j + 3] * s4.w * ex2(li - l4.w)};
            if (cg == q4) {
#pragma unroll
              for (int u = 0; u < 4; ++u) v[u] = j + u <= lane ? v[u] : 0.f;
            }
            m[hh][j / 2] = pack_bf16(v[0], v[1]);
            m[hh][j / 2 + 1] = pack_bf16(v[2], v[3]);
          }
        }
      } else {
#pragma unroll
        for (int hh = 0; hh < HPC; ++hh)
#pragma unroll
          for (int j = 0; j < 16; ++j) m[hh][j] = 0u;
      }
      // in the place of the scores that this thread has read: 16 columns a head
#pragma unroll
      for (int hh = 0; hh < HPC; ++hh) tmem_st16_nowait(tq + kColSc + 32 * cg + 16 * hh, m[hh]);
    }
    // ---- y = e^{L_i} (C S^T), in place ------------------------------------------------------------
    wait(b_in, par, 1);
    tc::fence_after();
    if (loader && c + 1 < nc) load_c(c + 1);
    __syncwarp();
    {
      float y[C::kYC];
      tmem_load<C::kYC>(tq + kColY + yc, y);
      const float e = exp2f(tab[yh * 3 * kQ + row]);
      uint32_t u[C::kYC];
#pragma unroll
      for (int i = 0; i < C::kYC; ++i) u[i] = __float_as_uint(e * y[i]);
#pragma unroll
      for (int i = 0; i < C::kYC; i += 16)
        tmem_st16_nowait(tq + kColY + yc + i, reinterpret_cast<const uint32_t(&)[16]>(u[i]));
    }
    // ---- w x of the other 64 tokens -----------------------------------------------------------------
    wait(b_d0, par, 1);
    tc::fence_after();
    if (32 * q4 < C::kRows) split_xw(xt, tab + hr * 3 * kQ + 2 * kQ, row, 64 + 16 * cg, tq + kColXw + 8 * cg);
    tmem_st_wait();
    tc::fence_before();
    __syncthreads();
    if (*abort_flag) { aborted = true; break; }
    if (issuer) {
      tc::fence_after();
      constexpr uint32_t kId = tc::idesc_bf16(128, PB, 0, 1);
#pragma unroll
      for (int hh = 0; hh < HPC; ++hh) {
        const uint64_t xd = tc::sdesc(sb + (c & 1) * C::kStage + C::kOffX + hh * 16384, 16384, 1024, tc::kSw128);
#pragma unroll
        for (int ks = 0; ks < kQ / 16; ++ks)
          tc::mma_f16_ta(tmem + kColY + hh * PB, tmem + kColSc + 32 * (ks >> 1) + 16 * hh + 8 * (ks & 1),
                         xd + (uint64_t)((ks * 2048) >> 4), kId, 1u);
      }
      tc::commit(b_y);
      issue_state<DK>(tmem, tmem + kColXw, sb + (c & 1) * C::kStage + C::kOffB, 1, false);
      tc::commit(b_d1);
    }
    __syncwarp();
    // every thread has stored the chunk before's outputs: its stage takes the chunk after this one
    if (loader && c > 0 && c + 1 < nc) load_stage(c + 1);
    __syncwarp();

    // ---- outputs, staged over the x tile -----------------------------------------------------------
    uint4 zr[C::kYC / 8];
    const bool gate = a.z != nullptr && my_cols && row < n;
    if (gate) {
      const __nv_bfloat16* zp = a.z + (tok0 + (long long)c * kQ + row) * a.zs + (h0 + yh) * a.dv + yp;
#pragma unroll
      for (int i = 0; i < C::kYC / 8; ++i) zr[i] = *reinterpret_cast<const uint4*>(zp + 8 * i);
    }
    wait(b_y, par, 1);
    tc::fence_after();
    if (issuer && c + 1 < nc) issue_scores(c + 1);  // the scores' place is free: M x is done
    __syncwarp();
    {
      float y[C::kYC];
      tmem_load<C::kYC>(tq + kColY + yc, y);
#pragma unroll
      for (int i = 0; i < C::kYC / 8; ++i) {
        uint4* at = reinterpret_cast<uint4*>(xt + ((yc + 8 * i) >> 6) * 16384 +
                                             tc::sw128((uint32_t)row, (uint32_t)((yc + 8 * i) & 63) >> 3));
        const uint4 xr = *at;
        const uint32_t xw4[4] = {xr.x, xr.y, xr.z, xr.w}, zw4[4] = {zr[i].x, zr[i].y, zr[i].z, zr[i].w};
        uint32_t o4[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          float v0 = fmaf(skip, __uint_as_float(xw4[u] << 16), y[8 * i + 2 * u]);
          float v1 = fmaf(skip, __uint_as_float(xw4[u] & 0xffff0000u), y[8 * i + 2 * u + 1]);
          if (gate) {
            v0 *= ssm_silu(__uint_as_float(zw4[u] << 16));
            v1 *= ssm_silu(__uint_as_float(zw4[u] & 0xffff0000u));
          }
          o4[u] = pack_bf16(v0, v1);
        }
        *at = make_uint4(o4[0], o4[1], o4[2], o4[3]);
      }
    }
    // ---- S = e^{L_last} S + the chunk's sum ---------------------------------------------------------
    wait(b_d1, par, 1);
    tc::fence_after();
    {
      float ds[C::kSC];
      tmem_load<C::kSC>(tq + kColDs + C::kSC * cg, ds);
      const SsmDecay decay = lend[(c & 1) * HPC + hr];
#pragma unroll
      for (int i = 0; i < C::kSC; ++i) st[i] = ssm_decayed(decay, st[i], ds[i]);
    }
    tc::fence_before();
  }
  __syncthreads();
  if (!aborted && *abort_flag) aborted = true;
  if (!aborted && nc > 0) copy_out(nc - 1);
  if (!aborted && fin != nullptr && s.last && my_row) {
    float* dst = fin + (((size_t)s.b * a.Hv + h0 + hr) * a.dv + p) * DK + C::kSC * cg;
#pragma unroll
    for (int i = 0; i < C::kSC; i += 4) *reinterpret_cast<float4*>(dst + i) = make_float4(st[i], st[i + 1], st[i + 2], st[i + 3]);
  }
  if (aborted && issuer) {  // let what is in flight land, bounded again, before the CTA leaves
    for (int i = 0; i < 8; ++i)
      for (uint32_t par = 0; par < 2; ++par) (void)tc::mbar_wait(&bars[i], par, 1u << 14);
  }
  tc::fence_before();
  __syncthreads();
  if (warp == 12) tc::tmem_dealloc(tmem, kTmemCols);
}

// The sums of the segments before a sequence's last (from a zero state) and their decays in log2.
// grid: segments x head blocks, the head blocks of a segment side by side (they read the same B and C).
template <int DK, int PB, int HPC>
__global__ void __launch_bounds__(kThreads, 1)
gdn_ssm_segment_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_b,
                       const SsmArgs a, const Segs g, float* __restrict__ seg_state, float* __restrict__ seg_decay,
                       int* __restrict__ err) {
  using C = Cfg<DK, PB, HPC>;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw_s = smem_u32(smem_raw);
  const uint32_t pad = ((raw_s + 1023u) & ~1023u) - raw_s;
  unsigned char* sm = smem_raw + pad;
  const uint32_t sb = raw_s + pad;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + C::kOffBar);
  uint64_t *b_d = bars, *b_st = bars + 1;  // the chunk's product; stage loaded (2)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  SsmDecay* lend = reinterpret_cast<SsmDecay*>(tmem_slot + 2);
  float* tabs = reinterpret_cast<float*>(sm + C::kOffTab);

  const int nhb = a.Hv / HPC, seg = blockIdx.x / nhb;
  Seg s;
  if (!find_seg(g, seg, s) || s.last) return;  // a last segment's sum is nobody's start
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int q4 = warp & 3, cg = warp >> 2;
  const int row = 32 * q4 + lane;
  const bool issuer = warp == 12 && lane == 0, loader = warp == 4 && lane == 0;
  const int tab_head = warp == 8 ? 0 : (HPC == 2 && warp == 13) ? 1 : -1;
  if (warp == 12) {
    tc::tmem_alloc(tmem_slot, kTmemCols);
    tc::tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < 3; ++i) tc::mbar_init(&bars[i], 1);
    tc::fence_mbar_init();
    *abort_flag = 0;
  }
  const int h0 = (blockIdx.x - seg * nhb) * HPC;
  const int hk = h0 / (a.Hv / a.Hk);
  const int nc = (s.t1 - s.t0) / kQ;  // whole chunks: only a last segment is ragged
  const long long tok0 = s.bos + s.t0;
  const int hr = HPC == 2 ? row >> 6 : 0, p = PB == 64 ? row & 63 : row;
  const bool my_row = row < C::kRows && p < a.dv;
  float st[C::kSC];
#pragma unroll
  for (int i = 0; i < C::kSC; ++i) st[i] = 0.f;

  auto load_stage = [&](int c) {
    unsigned char* dst = sm + (c & 1) * C::kStage;
    uint64_t* bar = &b_st[c & 1];
    const int t = (int)(tok0 + (long long)c * kQ);
    tc::mbar_arrive_expect_tx(bar, C::kStage);
#pragma unroll
    for (int i = 0; i < C::kNB; ++i) tc::tma_load_2d(dst + C::kOffB + i * 16384, &tm_b, hk * DK + 64 * i, t, bar);
#pragma unroll
    for (int i = 0; i < C::kXB; ++i)
      tc::tma_load_2d(dst + C::kOffX + i * 16384, &tm_x, PB == 64 ? (h0 + i) * a.dv : h0 * a.dv + 64 * i, t, bar);
  };
  auto wait = [&](uint64_t* bar, uint32_t par, int bit) {
    if (!tc::mbar_wait(bar, par, kMaxPolls)) {
      *abort_flag = 1;
      atomicOr(err, bit);
    }
  };
  float d[4] = {0.f, 0.f, 0.f, 0.f}, total = 0.f;
  const float a_log2 = tab_head >= 0 ? a.A[h0 + tab_head] * 1.4426950408889634f : 0.f;
  auto tables = [&](int c) {
    const float end = make_tables<true>(tabs + (c & 1) * (C::kTab / 4) + tab_head * kQ, d, a_log2, lane);
    total += end;
    if (lane == 0) lend[(c & 1) * HPC + tab_head] = ssm_decay(end * 0.6931471805599453f);
    if (c + 1 < nc) load_steps(a, tok0 + (long long)(c + 1) * kQ, kQ, h0 + tab_head, lane, d);
  };
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tq = tmem + ((uint32_t)(32 * q4) << 16);
  if (loader) {
    load_stage(0);
    if (nc > 1) load_stage(1);
  }
  if (tab_head >= 0) {
    load_steps(a, tok0, kQ, h0 + tab_head, lane, d);
    tables(0);
  }
  __syncthreads();
  bool aborted = false;
  // w x of a chunk (both halves) in two buffers over the columns that outputs would take: 0.. and 128..,
  // 96 columns a half at 0, 96 | 384, 256 + 128
  auto xw_col = [](int c, int hf) { return (uint32_t)((c & 1) ? (hf ? 416 : 192) : (hf ? 96 : 0)); };
  auto update = [&](int c) {  // S after chunk c, whose product is awaited
    wait(b_d, (uint32_t)(c & 1), 1);
    tc::fence_after();
    float ds[C::kSC];
    tmem_load<C::kSC>(tq + 288 + C::kSC * cg, ds);
    const SsmDecay decay = lend[(c & 1) * HPC + hr];
#pragma unroll
    for (int i = 0; i < C::kSC; ++i) st[i] = ssm_decayed(decay, st[i], ds[i]);
  };
  for (int c = 0; c < nc; ++c) {
    const float* w = tabs + (c & 1) * (C::kTab / 4) + hr * kQ;
    const unsigned char* xt = sm + (c & 1) * C::kStage + C::kOffX;
    wait(&b_st[c & 1], (uint32_t)((c >> 1) & 1), 2);
    if (32 * q4 < C::kRows) {
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) split_xw(xt, w, row, 64 * hf + 16 * cg, tq + xw_col(c, hf) + 8 * cg);
    }
    if (c > 0) update(c - 1);
    tmem_st_wait();
    tc::fence_before();
    __syncthreads();  // the tables of c - 1 and its stage are free, the sum of c - 1 has been read
    if (*abort_flag) { aborted = true; break; }
    if (issuer) {
      tc::fence_after();
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
        issue_state<DK>(tmem + 288 - kColDs, tmem + xw_col(c, hf), sb + (c & 1) * C::kStage + C::kOffB, hf, hf == 0);
      tc::commit(b_d);
    }
    __syncwarp();
    if (loader && c > 0 && c + 1 < nc) load_stage(c + 1);
    __syncwarp();
    if (tab_head >= 0 && c + 1 < nc) tables(c + 1);
    __syncthreads();  // the next tables
  }
  if (!aborted) update(nc - 1);
  __syncthreads();
  if (*abort_flag) aborted = true;
  if (!aborted && my_row) {
    float* dst = seg_state + (((size_t)s.slot * a.Hv + h0 + hr) * a.dv + p) * DK + C::kSC * cg;
#pragma unroll
    for (int i = 0; i < C::kSC; i += 4) *reinterpret_cast<float4*>(dst + i) = make_float4(st[i], st[i + 1], st[i + 2], st[i + 3]);
  }
  if (!aborted && tab_head >= 0 && lane == 0) seg_decay[(size_t)s.slot * a.Hv + h0 + tab_head] = total;
  if (aborted && issuer) {
    for (int i = 0; i < 3; ++i)
      for (uint32_t par = 0; par < 2; ++par) (void)tc::mbar_wait(&bars[i], par, 1u << 14);
  }
  tc::fence_before();
  __syncthreads();
  if (warp == 12) tc::tmem_dealloc(tmem, kTmemCols);
}

template <int DK, int PB, int HPC>
cudaError_t launch(const CUtensorMap& tx, const CUtensorMap& tb, const CUtensorMap& tcm, const SsmArgs& a,
                   const Segs& g, float* seg_state, float* seg_decay, const float* init, float* fin, int* err,
                   int phase, cudaStream_t st) {
  using C = Cfg<DK, PB, HPC>;
  const unsigned grid = (unsigned)(a.Hv / HPC) * (unsigned)g.slots;
  if (phase == 0) {
    const cudaError_t e = set_smem_limit_once<gdn_ssm_segment_kernel<DK, PB, HPC>>(C::kSmemBytes);
    if (e != cudaSuccess) return e;
    gdn_ssm_segment_kernel<DK, PB, HPC><<<grid, kThreads, C::kSmemBytes, st>>>(tx, tb, a, g, seg_state, seg_decay, err);
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
  e = cudaLaunchKernelEx(&cfg, gdn_ssm_chunk_kernel<DK, PB, HPC>, tx, tb, tcm, a, g, (const float*)seg_state, init, fin,
                         err);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

template <int DK>
cudaError_t launch_dk(const CUtensorMap& tx, const CUtensorMap& tb, const CUtensorMap& tcm, const SsmArgs& a,
                      const Segs& g, float* seg_state, float* seg_decay, const float* init, float* fin, int* err,
                      int hpc, int phase, cudaStream_t st) {
  if (a.dv == 128) return launch<DK, 128, 1>(tx, tb, tcm, a, g, seg_state, seg_decay, init, fin, err, phase, st);
  if (hpc == 2) return launch<DK, 64, 2>(tx, tb, tcm, a, g, seg_state, seg_decay, init, fin, err, phase, st);
  return launch<DK, 64, 1>(tx, tb, tcm, a, g, seg_state, seg_decay, init, fin, err, phase, st);
}

}  // namespace ssm
}  // namespace gdn
