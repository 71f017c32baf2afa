// Launches of the selective state space scan of a prompt (gdn_ssm_chunk.cuh): tensor maps, the choice of
// segments, and the pass that joins them.
//
// A CTA carries the state of its heads through a segment's chunks one after the other.  Where sequences
// and heads are too few to fill the device, sequences are cut into segments: one pass sums every segment
// from a zero state (x, B and dt only, about 0.3 of a chunk's time), and the output pass runs every segment
// from the sums before it (with many segments gdn_ssm_join_kernel makes start states of them first).  The
// later kernels are programmatic dependents: they set up beside the one before.
#include <algorithm>
#include <atomic>

#include "../../include/gdn.h"
#include "gdn_internal.h"
#include "gdn_ssm_chunk.cuh"

namespace gdn {

cudaError_t launch_chunk_table(const int32_t*, int, int, int32_t*, int32_t*, int*, cudaStream_t);

namespace ssm {
template <int DK>
cudaError_t launch_dk(const Maps&, const SsmArgs&, const Segs&, float*, float*, const float*, float*, float*, int*, int,
                      int, cudaStream_t);
}

namespace {

constexpr int kJoinThreads = 128;
constexpr int kAloneSegs = 8;  // segments a sequence that the output pass goes through by itself

std::atomic<int> g_polls{(int)ssm::kMaxPolls};

struct Plan {
  int hpc = 1;    // heads a CTA
  int len = 0;    // chunks a segment (0: whole sequences)
  int slots = 0;  // segments
};

// Heads a CTA and the segments' length, from the sizes alone (a packed batch's lengths are on the device:
// taken as equal).  In units of an output pass's chunk step (4.2 us at 128 x 128): a CTA costs its chunks and about one
// more to start and drain, 0.25 of a step a chunk and 0.8 in the pass of the sums, and the join about one.  The choice
// does not hang on these (from 0.1 to 0.6 of a step a chunk it is the same for 1,024, 4,096 and 16,381 tokens).
Plan make_plan(int B, int T, int Hk, int Hv, int dv, bool packed, int sms) {
  Plan p;
  p.hpc = dv < 128 && (Hv / Hk) % 2 == 0 ? 2 : 1;
  const long long hb = Hv / p.hpc;
  p.slots = B;
  if (B == 0 || T == 0) return p;
  const int nc = (int)(((packed ? ((long long)T + B - 1) / B : (long long)T) + ssm::kQ - 1) / ssm::kQ);
  auto waves = [&](long long ctas) { return (ctas + sms - 1) / sms; };
  double best = (double)waves(hb * B) * (nc + 1);
  for (int n = 2; n <= nc; ++n) {  // segments a sequence
    const int len = (nc + n - 1) / n;
    if (n > 2 && (nc + n - 2) / (n - 1) == len) continue;  // the same length as with fewer
    const long long segs = (nc + len - 1) / len;
    const double cost = waves(hb * B * segs) * (len + 1.0) +
                        waves(hb * B * (segs - 1)) * (0.25 * len + 0.8) + (segs > kAloneSegs ? 1.0 : 0.15 * (segs - 1));
    if (cost < best) {
      best = cost;
      p.len = len;
    }
    if (hb * B * segs > 4LL * sms) break;
  }
  if (p.len != 0) {
    const int per = p.len * ssm::kQ;
    p.slots = packed ? T / per + B : B * ((T - 1) / per + 1);
  }
  return p;
}

// The segments' sums E_k joined, in place: the state before segment k but for the initial state, and the log of that
// state's decay up to it.  One thread per four values of a (sequence, head block), in the workspace's layout by
// worker threads (`pb` rows reserved for each of `hpc` heads).  grid: (B * head blocks, blocks over dk * 32)
__global__ void __launch_bounds__(kJoinThreads)
gdn_ssm_join_kernel(const ssm::Segs g, float* __restrict__ seg_state, const float* __restrict__ seg_decay,
                    float* __restrict__ seg_total, int Hv, int dk, int dv, int pb, int hpc) {
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const int nhb = Hv / hpc, b = blockIdx.x / nhb, hb = blockIdx.x - b * nhb;
  const int e = blockIdx.y * kJoinThreads + threadIdx.x;
  const int worker = e % (32 * ssm::kWorkers), row = 32 * ((worker >> 5) & 3) + (worker & 31);
  const int hr = hpc == 2 ? row >> 6 : 0, p = pb == 64 ? row & 63 : row;
  int slot0 = 0, n;
  if (g.cu == nullptr) {
    n = ssm::seg_count(g, g.T);
    slot0 = b * n;
  } else {
    n = ssm::seg_count(g, seq_bounds(g.cu, b, g.T).len);
    const int lane = threadIdx.x & 31;  // segments of the sequences before: every warp sums them
    long long sum = 0;
    for (int i = lane; i < b; i += 32) sum += ssm::seg_count(g, seq_bounds(g.cu, i, g.T).len);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    slot0 = sum < g.slots ? (int)sum : g.slots;  // malformed boundaries may claim more than there are
    n = n < g.slots - slot0 ? n : g.slots - slot0;
  }
  if (e >= dk * 32 || row >= pb * hpc || p >= dv) return;
  const int h = hb * hpc + hr;
  const bool teller = p == 0 && worker < 32 * 4 && e == worker;  // one thread a head
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  float total = 0.f;
  constexpr int kAhead = 16;
  float4 v[kAhead];
  float l[kAhead];
  auto at = [&](int k) {
    return reinterpret_cast<float4*>(seg_state) + ((size_t)(slot0 + k) * nhb + hb) * dk * 32 + e;
  };
  for (int k0 = 0; k0 < n; k0 += kAhead) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (k0 + u + 1 < n) {
        v[u] = *at(k0 + u);
        l[u] = seg_decay[(size_t)(slot0 + k0 + u) * Hv + h];
      }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (k0 + u >= n) break;
      if (k0 + u > 0) *at(k0 + u) = s;
      if (teller) seg_total[(size_t)(slot0 + k0 + u) * Hv + h] = total;
      if (k0 + u + 1 < n) {
        const SsmDecay m = ssm_decay(l[u] * 0.6931471805599453f);
        total += l[u];
        s.x = ssm_decayed(m, s.x, v[u].x);
        s.y = ssm_decayed(m, s.y, v[u].y);
        s.z = ssm_decayed(m, s.z, v[u].z);
        s.w = ssm_decayed(m, s.w, v[u].w);
      }
    }
  }
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// Workspace: [256 B status words][packed: chunk table and dispatch order][segment states, 128 rows a head block]
//            [segment decays][joined decays][copy of the initial states]
struct Layout {
  size_t states, decays, totals, kept, total;
};
Layout layout(const Plan& p, int B, int Hv, int dk, int dv, bool packed) {
  Layout l;
  l.states = 256 + (packed ? chunk_table_bytes(B) : 0);
  const size_t n = p.len != 0 ? (size_t)p.slots : 0;
  l.decays = l.states + align256(n * (Hv / p.hpc) * dk * 128 * 4);
  l.totals = l.decays + align256(n * Hv * 4);
  l.kept = l.totals + align256(n * Hv * 4);
  l.total = l.kept + (p.len != 0 ? align256((size_t)B * Hv * dv * dk * 4) : 0);
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

int ssm_scan_polls(int polls) { return g_polls.exchange(polls < 0 ? (int)ssm::kMaxPolls : polls); }

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
  float* totals = reinterpret_cast<float*>(w + l.totals);
  // In place, a sequence's last segment may end before an earlier one has read the initial state.
  float* kept = p.len != 0 && init != nullptr && init == fin ? reinterpret_cast<float*>(w + l.kept) : nullptr;
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
  g.polls = (uint32_t)g_polls.load(std::memory_order_relaxed);
  // With few segments a sequence the output pass goes through the sums before its own by itself (about 0.8 us each,
  // beside its first tiles' load); more are joined by a kernel (10 us by itself for 32 segments).
  const int per = p.len * ssm::kQ;
  g.joined = p.len != 0 && (T - 1) / per + 1 > kAloneSegs;
  auto run = [&](int phase) {
    float* dec = phase == 1 && g.joined ? totals : decays;
    switch (dk) {
      case 32: return ssm::launch_dk<32>(m, a, g, states, dec, init, kept, fin, err, p.hpc, phase, st);
      case 64: return ssm::launch_dk<64>(m, a, g, states, dec, init, kept, fin, err, p.hpc, phase, st);
      default: return ssm::launch_dk<128>(m, a, g, states, dec, init, kept, fin, err, p.hpc, phase, st);
    }
  };
  cudaError_t e;
  if (p.len != 0) {
    if ((e = run(0)) != cudaSuccess) return e;
  }
  if (g.joined) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(B * (a.Hv / p.hpc)), (unsigned)(dk * 32 / kJoinThreads));
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, gdn_ssm_join_kernel, (const ssm::Segs)g, states, (const float*)decays, totals, a.Hv,
                           dk, a.dv, a.dv == 128 ? 128 : 64, p.hpc);
    if (e != cudaSuccess) return e;
  } else if (p.len == 0 && packed && B > 1) {  // whole sequences of different lengths: the longest start first
    int32_t* off = reinterpret_cast<int32_t*>(w + 256);
    if ((e = launch_chunk_table(cu, B, T, off, off + B + 1, err, st)) != cudaSuccess) return e;
    g.order = off + B + 1;
  }
  return run(1);
}

}  // namespace gdn
