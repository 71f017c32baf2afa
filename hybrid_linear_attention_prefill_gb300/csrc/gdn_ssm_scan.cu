// Launches of the selective state space scan of a prompt (gdn_ssm_chunk.cuh): tensor maps, the choice of
// segments, and the pass that joins them.
//
// A CTA carries the state of its heads through a segment's chunks one after the other.  Where sequences
// and heads are too few to fill the device, sequences are cut into segments: one pass sums every segment
// from a zero state (x, B and dt only, about 0.4 of a chunk's time), gdn_ssm_join_kernel turns the sums
// into start states, and the output pass runs every segment from its own.
#include <algorithm>

#include "../../include/gdn.h"
#include "gdn_internal.h"
#include "gdn_ssm_chunk.cuh"

namespace gdn {

cudaError_t launch_chunk_table(const int32_t*, int, int, int32_t*, int32_t*, int*, cudaStream_t);

namespace ssm {
template <int DK>
cudaError_t launch_dk(const Maps&, const SsmArgs&, const Segs&, float*, float*, const float*, float*, int*, int, int,
                      cudaStream_t);
}

namespace {

constexpr int kJoinThreads = 256;

struct Plan {
  int hpc = 1;    // heads a CTA
  int len = 0;    // chunks a segment (0: whole sequences)
  int slots = 0;  // segments
};

// Heads a CTA and the segments' length, from the sizes alone (a packed batch's lengths are on the device:
// taken as equal).  In units of an output pass's chunk step: a CTA costs its chunks and about one more to start
// and drain, 0.4 of a step a chunk and one in the pass of the sums, and the join about one.
Plan make_plan(int B, int T, int Hk, int Hv, int dv, bool packed, int sms) {
  Plan p;
  p.hpc = dv < 128 && (Hv / Hk) % 2 == 0 ? 2 : 1;
  const long long hb = Hv / p.hpc;
  p.slots = B;
  if (B == 0 || T == 0) return p;
  const int nc = packed ? std::max(1, (int)(((long long)T + B - 1) / B + ssm::kQ - 1) / ssm::kQ)
                        : (T + ssm::kQ - 1) / ssm::kQ;
  auto waves = [&](long long ctas) { return (ctas + sms - 1) / sms; };
  double best = (double)waves(hb * B) * (nc + 1);
  for (int n = 2; n <= nc; ++n) {  // segments a sequence
    const int len = (nc + n - 1) / n;
    if (n > 2 && (nc + n - 2) / (n - 1) == len) continue;  // the same length as with fewer
    const long long segs = (nc + len - 1) / len;
    const double cost = waves(hb * B * segs) * (len + 1.0) + waves(hb * B * (segs - 1)) * (0.4 * len + 1.0) + 1.0;
    if (cost < best) {
      best = cost;
      p.len = len;
    }
    if (hb * B * segs > 4LL * sms) break;
  }
  if (p.len != 0) {
    const int per = p.len * ssm::kQ;
    p.slots = packed ? T / per + B : B * ((T + per - 1) / per);
  }
  return p;
}

// Segment start states from the segments' sums E and decays, in place: S_start(0) = the initial state,
// S_start(k + 1) = decay_k S_start(k) + E_k.  One thread per four state elements of a (sequence, head).
// grid: (B * Hv, blocks over dv * dk / 4)
__global__ void __launch_bounds__(kJoinThreads)
gdn_ssm_join_kernel(const ssm::Segs g, const float* __restrict__ init, float* __restrict__ seg_state,
                    const float* __restrict__ seg_decay, int Hv, int nstate) {
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const int b = blockIdx.x / Hv, h = blockIdx.x - b * Hv;
  const int e = blockIdx.y * kJoinThreads + threadIdx.x;
  int slot0 = 0, n;
  if (g.cu == nullptr) {
    n = ssm::seg_count(g, g.T);
    slot0 = b * n;
  } else {
    n = ssm::seg_count(g, seq_bounds(g.cu, b, g.T).len);
    const int lane = threadIdx.x & 31;  // segments of the sequences before: every warp sums them
    int sum = 0;
    for (int i = lane; i < b; i += 32) sum += ssm::seg_count(g, seq_bounds(g.cu, i, g.T).len);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    slot0 = sum;
    if (slot0 > g.slots) slot0 = g.slots;
    if (n > g.slots - slot0) n = g.slots - slot0;  // malformed boundaries
  }
  if (4 * e >= nstate) return;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (init != nullptr) s = *reinterpret_cast<const float4*>(init + ((size_t)b * Hv + h) * nstate + 4 * e);
  constexpr int kAhead = 4;
  float4 v[kAhead];
  SsmDecay m[kAhead];
  auto at = [&](int k) { return seg_state + ((size_t)(slot0 + k) * Hv + h) * nstate + 4 * e; };
  for (int k0 = 0; k0 < n; k0 += kAhead) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (k0 + u + 1 < n) {
        v[u] = *reinterpret_cast<const float4*>(at(k0 + u));
        m[u] = ssm_decay(seg_decay[(size_t)(slot0 + k0 + u) * Hv + h] * 0.6931471805599453f);
      }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (k0 + u >= n) break;
      *reinterpret_cast<float4*>(at(k0 + u)) = s;
      if (k0 + u + 1 < n) {
        s.x = ssm_decayed(m[u], s.x, v[u].x);
        s.y = ssm_decayed(m[u], s.y, v[u].y);
        s.z = ssm_decayed(m[u], s.z, v[u].z);
        s.w = ssm_decayed(m[u], s.w, v[u].w);
      }
    }
  }
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// Workspace: [256 B status words][packed: chunk table and dispatch order][segment states][segment decays]
struct Layout {
  size_t states, decays, total;
};
Layout layout(const Plan& p, int B, int Hv, int dk, int dv, bool packed) {
  Layout l;
  l.states = 256 + (packed ? chunk_table_bytes(B) : 0);
  const size_t n = p.len != 0 ? (size_t)p.slots * Hv : 0;
  l.decays = l.states + align256(n * dv * dk * 4);
  l.total = l.decays + align256(n * 4);
  return l;
}

bool token_map(CUtensorMap* m, const void* base, long long stride, long long width, long long tokens,
               cuuint32_t box_tokens = ssm::kQ) {
  const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)tokens};
  const cuuint64_t strides[1] = {(cuuint64_t)(tokens > 1 ? stride : (width + 7) / 8 * 8) * 2};
  const cuuint32_t box[2] = {64, box_tokens};
  return make_map16(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, 2, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace

size_t ssm_scan_workspace(int B, int T, int Hk, int Hv, int dk, int dv, int packed) {
  const int sms = device_sms();
  // without a device: enough for any (a segment of one chunk for every chunk)
  Plan p = make_plan(B, T, Hk, Hv, dv, packed != 0, sms > 0 ? sms : 1 << 20);
  return layout(p, B, Hv, dk, dv, packed != 0).total;
}

cudaError_t launch_ssm_scan(const SsmArgs& a, const int32_t* cu, const float* init, float* fin, void* ws, int B, int T,
                            int dk, cudaStream_t st) {
  const int sms = device_sms();
  if (sms == 0) return cudaErrorNoDevice;
  const bool packed = cu != nullptr;
  const Plan p = make_plan(B, T, a.Hk, a.Hv, a.dv, packed, sms);
  const Layout l = layout(p, B, a.Hv, dk, a.dv, packed);
  unsigned char* w = static_cast<unsigned char*>(ws);
  int* err = static_cast<int*>(ws);
  float* states = reinterpret_cast<float*>(w + l.states);
  float* decays = reinterpret_cast<float*>(w + l.decays);
  const long long ntok = packed ? (long long)T : (long long)B * T;
  if ((long long)p.slots * (a.Hv / p.hpc) > 0x7fffffffLL) return cudaErrorInvalidValue;
  ssm::Maps m = {};
  const long long wv = (long long)a.Hv * a.dv, wk = (long long)a.Hk * dk;
  if (ntok > 0 &&
      (!token_map(&m.x, a.x, a.xs, wv, ntok) || !token_map(&m.b, a.Bm, a.bs, wk, ntok) ||
       !token_map(&m.c, a.Cm, a.cs, wk, ntok) || (a.z != nullptr && !token_map(&m.z, a.z, a.zs, wv, ntok)) ||
       !token_map(&m.out, a.out, wv, wv, ntok, 32)))
    return cudaErrorInvalidValue;
  ssm::Segs g;
  g.cu = cu;
  g.order = nullptr;
  g.B = B;
  g.T = T;
  g.len = p.len;
  g.slots = p.slots;
  auto run = [&](int phase) {
    switch (dk) {
      case 32: return ssm::launch_dk<32>(m, a, g, states, decays, init, fin, err, p.hpc, phase, st);
      case 64: return ssm::launch_dk<64>(m, a, g, states, decays, init, fin, err, p.hpc, phase, st);
      default: return ssm::launch_dk<128>(m, a, g, states, decays, init, fin, err, p.hpc, phase, st);
    }
  };
  cudaError_t e;
  if (p.len != 0) {
    if ((e = run(0)) != cudaSuccess) return e;
    const int nstate = a.dv * dk;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(B * a.Hv), (unsigned)((nstate / 4 + kJoinThreads - 1) / kJoinThreads));
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, gdn_ssm_join_kernel, (const ssm::Segs)g, init, states, (const float*)decays, a.Hv, nstate);
    if (e != cudaSuccess) return e;
  } else if (packed && B > 1) {  // whole sequences of different lengths: the longest start first
    int32_t* off = reinterpret_cast<int32_t*>(w + 256);
    if ((e = launch_chunk_table(cu, B, T, off, off + B + 1, err, st)) != cudaSuccess) return e;
    g.order = off + B + 1;
  }
  return run(1);
}

}  // namespace gdn
