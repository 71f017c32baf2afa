// C ABI of attention and its paged key-value cache.  Argument checks here, kernels in gdn_cache.cu,
// gdn_attn.cu and gdn_attn_step.cu.
#include <cmath>

#include "gdn_args.h"
#include "gdn_attn.cuh"
#include "gdn_cache.h"

namespace gdn {
cudaError_t launch_attn(const attn::PromptArgs&, int*, cudaStream_t);
cudaError_t launch_attn_step(const attn::StepArgs&, bool, void*, int*, cudaStream_t);
size_t attn_step_workspace(int, int, int, int);
}  // namespace gdn

namespace {

using gdn::aligned;
using gdn::check_rows;
using gdn::done;
using gdn::overlap;

bool heads_ok(int Hq, int Hkv, int d) {
  return Hkv > 0 && Hq > 0 && Hq % Hkv == 0 && Hq <= 65535 && d > 0 && d % 8 == 0 && d <= gdn::attn::kMaxDim;
}

bool page_ok(int page, int blocks) {
  return page > 0 && page % 16 == 0 && blocks >= 0 && (long long)page * blocks <= 0x7fffffffLL;
}

// A cache whose blocks are contiguous: GDN_OK, or what is wrong with it.
int check_cache(const void* p, long long stride, int Hkv, int d, int page, int blocks) {
  if (p == nullptr || (blocks > 1 && stride < (long long)Hkv * page * d)) return GDN_ERR_ARG;
  if (!aligned(p, 16) || (blocks > 1 && stride % 16 != 0)) return GDN_ERR_ALIGN;
  return GDN_OK;
}

// The call's workspace of `need` bytes: the given one, whose first word is for status bits, or the library's own, of which
// `status_only` wants no more than those.
int workspace_for(void* given, size_t given_bytes, size_t need, bool status_only, void* stream, gdn::AttnOwn& own) {
  if (given != nullptr) {
    if (!aligned(given, 256)) return GDN_ERR_ALIGN;
    if (given_bytes < need) return GDN_ERR_SCRATCH;
    own.ws = given;
    own.status = static_cast<int*>(given);
    return GDN_OK;
  }
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return gdn::set_cuda_error(e, GDN_ERR_LAUNCH);
  return gdn::own_attn_workspace(dev, status_only ? 0 : need, static_cast<cudaStream_t>(stream), own);
}

}  // namespace

extern "C" {

int gdn_cache_plan(const gdn_cache_plan_args* args) {
  gdn::clear_cuda_error();
  if (args == nullptr) return GDN_ERR_ARG;
  const auto& [lens, block_table, table_stride, free_blocks, free_count, cu_seqlens, slots, new_lens, new_count, refused,
               B, T, W, capacity, page, stream] = *args;
  if (B < 0 || T < 0 || W < 0 || capacity < 0 || B > gdn::kPlanMaxRequests || !page_ok(page, 0)) return GDN_ERR_ARG;
  if (cu_seqlens == nullptr && T != B) return GDN_ERR_ARG;
  if (free_count == nullptr || new_count == nullptr || (capacity > 0 && free_blocks == nullptr) ||
      (T > 0 && slots == nullptr))
    return GDN_ERR_ARG;
  if (B > 0 && (lens == nullptr || new_lens == nullptr || (W > 0 && block_table == nullptr))) return GDN_ERR_ARG;
  if (B > 1 && table_stride < W) return GDN_ERR_ARG;
  for (const void* p : {(const void*)lens, (const void*)block_table, (const void*)free_blocks, (const void*)free_count,
                        (const void*)cu_seqlens, (const void*)slots, (const void*)new_lens, (const void*)new_count,
                        (const void*)refused})
    if (!aligned(p, 4)) return GDN_ERR_ALIGN;
  gdn::CachePlanArgs a;
  a.lens = lens;
  a.table = block_table;
  a.table_stride = table_stride;
  a.free_blocks = free_blocks;
  a.free_count = free_count;
  a.cu = cu_seqlens;
  a.slots = slots;
  a.new_lens = new_lens;
  a.new_count = new_count;
  a.refused = refused;
  a.B = B;
  a.T = T;
  a.W = W;
  a.capacity = capacity;
  a.page = page;
  return done(gdn::launch_cache_plan(a, static_cast<cudaStream_t>(stream)));
}

int gdn_cache_append(const gdn_cache_append_args* args) {
  gdn::clear_cuda_error();
  if (args == nullptr) return GDN_ERR_ARG;
  const auto& [k, k_stride, v, v_stride, k_cache, k_block_stride, v_cache, v_block_stride, k_scale, v_scale, slots, T,
               Hkv, d, page, blocks, flags, stream] = *args;
  const bool e4m3 = (flags & GDN_CACHE_E4M3) != 0;
  if (T < 0 || !heads_ok(Hkv, Hkv, d) || !page_ok(page, blocks) || (flags & ~GDN_CACHE_E4M3) != 0) return GDN_ERR_ARG;
  if (T == 0 || blocks == 0) return GDN_OK;
  if (slots == nullptr || e4m3 != (k_scale != nullptr) || e4m3 != (v_scale != nullptr)) return GDN_ERR_ARG;
  int rc;
  if ((rc = check_rows(k, k_stride, T, (long long)Hkv * d)) != GDN_OK ||
      (rc = check_rows(v, v_stride, T, (long long)Hkv * d)) != GDN_OK ||
      (rc = check_cache(k_cache, k_block_stride, Hkv, d, page, blocks)) != GDN_OK ||
      (rc = check_cache(v_cache, v_block_stride, Hkv, d, page, blocks)) != GDN_OK)
    return rc;
  if (!aligned(slots, 4) || !aligned(k_scale, 4) || !aligned(v_scale, 4)) return GDN_ERR_ALIGN;
  gdn::CacheAppendArgs a;
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.ks = k_stride;
  a.vs = v_stride;
  a.kc = k_cache;
  a.vc = v_cache;
  a.kbs = k_block_stride;
  a.vbs = v_block_stride;
  a.kscale = k_scale;
  a.vscale = v_scale;
  a.slots = slots;
  a.T = T;
  a.Hkv = Hkv;
  a.d = d;
  a.page = page;
  a.blocks = blocks;
  return done(gdn::launch_cache_append(a, e4m3, static_cast<cudaStream_t>(stream)));
}

size_t gdn_attn_workspace_bytes(int B, int Hq, int Hkv, int d) {
  if (B < 0 || !heads_ok(Hq, Hkv, d)) return 0;
  return gdn::attn_step_workspace(B, Hq, Hkv, d);
}

int gdn_attn(const gdn_attn_args* args) {
  gdn::clear_cuda_error();
  if (args == nullptr) return GDN_ERR_ARG;
  const auto& [q, q_stride, k, k_stride, v, v_stride, cu_seqlens, cu_seqlens_k, out, lse, B, T, Tk, Hq, Hkv, d, window,
               sinks, scale, flags, given, given_bytes, stream] = *args;
  if (B < 0 || T < 0 || Tk < 0 || !heads_ok(Hq, Hkv, d) || Hq / Hkv > 128 || flags != 0) return GDN_ERR_ARG;
  if (window < 0 || sinks < 0 || !std::isfinite(scale)) return GDN_ERR_ARG;
  if (cu_seqlens == nullptr && cu_seqlens_k != nullptr) return GDN_ERR_ARG;
  if (cu_seqlens != nullptr && cu_seqlens_k == nullptr && T != Tk) return GDN_ERR_ARG;
  if (B == 0) return GDN_OK;
  const bool packed = cu_seqlens != nullptr;
  const long long nq = packed ? (long long)T : (long long)B * T, nk = packed ? (long long)Tk : (long long)B * Tk;
  if (nq > 0x7ffffc00LL || nk > 0x7ffffc00LL) return GDN_ERR_ARG;  // (a tile past the last token stays below 2^31)
  if (nq == 0) return GDN_OK;
  const long long wq = (long long)Hq * d, wk = (long long)Hkv * d;
  if (out == nullptr) return GDN_ERR_ARG;
  int rc;
  if ((rc = check_rows(q, q_stride, nq, wq)) != GDN_OK) return rc;
  if (nk > 0 && ((rc = check_rows(k, k_stride, nk, wk)) != GDN_OK || (rc = check_rows(v, v_stride, nk, wk)) != GDN_OK))
    return rc;
  if (!aligned(out, 16) || !aligned(lse, 4) || !aligned(cu_seqlens, 4) || !aligned(cu_seqlens_k, 4))
    return GDN_ERR_ALIGN;
  const size_t no = (size_t)nq * wq * 2;
  if (overlap(q, ((size_t)(nq - 1) * q_stride + wq) * 2, out, no)) return GDN_ERR_ARG;
  if (nk > 0 && (overlap(k, ((size_t)(nk - 1) * k_stride + wk) * 2, out, no) ||
                 overlap(v, ((size_t)(nk - 1) * v_stride + wk) * 2, out, no)))
    return GDN_ERR_ARG;
  gdn::AttnOwn own;
  if ((rc = workspace_for(given, given_bytes, 256, true, stream, own)) != GDN_OK) return rc;
  gdn::attn::PromptArgs a;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.qs = q_stride;
  a.ks = k_stride;
  a.vs = v_stride;
  a.cu = cu_seqlens;
  a.cuk = cu_seqlens_k != nullptr ? cu_seqlens_k : cu_seqlens;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.B = B;
  a.T = T;
  a.Tk = Tk;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.d = d;
  a.view = {window, sinks};
  a.scale = scale;
  return done(gdn::launch_attn(a, own.status, static_cast<cudaStream_t>(stream)));
}

int gdn_attn_step(const gdn_attn_step_args* args) {
  gdn::clear_cuda_error();
  if (args == nullptr) return GDN_ERR_ARG;
  const auto& [q, q_stride, k_cache, k_block_stride, v_cache, v_block_stride, k_scale, v_scale, block_table, table_stride,
               lens, out, lse, B, Hq, Hkv, d, page, blocks, W, window, sinks, scale, flags, given, given_bytes, stream] =
      *args;
  const bool e4m3 = (flags & GDN_CACHE_E4M3) != 0;
  if (B < 0 || W < 0 || !heads_ok(Hq, Hkv, d) || !page_ok(page, blocks) || (flags & ~GDN_CACHE_E4M3) != 0)
    return GDN_ERR_ARG;
  if (window < 0 || sinks < 0 || !std::isfinite(scale) || (long long)W * page > 0x7fffffffLL) return GDN_ERR_ARG;
  if (B == 0) return GDN_OK;
  if (lens == nullptr || out == nullptr || e4m3 != (k_scale != nullptr) || e4m3 != (v_scale != nullptr))
    return GDN_ERR_ARG;
  if (W > 0 && (block_table == nullptr || (B > 1 && table_stride < W))) return GDN_ERR_ARG;
  int rc;
  if ((rc = check_rows(q, q_stride, B, (long long)Hq * d)) != GDN_OK) return rc;
  if (blocks > 0 && ((rc = check_cache(k_cache, k_block_stride, Hkv, d, page, blocks)) != GDN_OK ||
                     (rc = check_cache(v_cache, v_block_stride, Hkv, d, page, blocks)) != GDN_OK))
    return rc;
  if (!aligned(out, 16) || !aligned(lse, 4) || !aligned(lens, 4) || !aligned(block_table, 4) || !aligned(k_scale, 4) ||
      !aligned(v_scale, 4))
    return GDN_ERR_ALIGN;
  if (overlap(q, ((size_t)(B - 1) * q_stride + (size_t)Hq * d) * 2, out, (size_t)B * Hq * d * 2)) return GDN_ERR_ARG;
  gdn::AttnOwn own;
  if ((rc = workspace_for(given, given_bytes, gdn::attn_step_workspace(B, Hq, Hkv, d), false, stream, own)) != GDN_OK)
    return rc;
  gdn::attn::StepArgs a;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.qs = q_stride;
  a.kc = k_cache;
  a.vc = v_cache;
  a.kbs = k_block_stride;
  a.vbs = v_block_stride;
  a.kscale = k_scale;
  a.vscale = v_scale;
  a.table = block_table;
  a.table_stride = table_stride;
  a.lens = lens;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.d = d;
  a.page = page;
  a.blocks = blocks;
  a.W = W;
  a.view = {window, sinks};
  a.scale = scale;
  return done(gdn::launch_attn_step(a, e4m3, own.ws, own.status, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
