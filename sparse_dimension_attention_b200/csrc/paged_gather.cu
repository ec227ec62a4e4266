// Pages of the 8-bit cache back into a contiguous f32 or bf16 cache: every code
// times its page's scale, keys dimension-major, values token-major.
//
// A copy bound by memory: (m + 128) bytes read and 2 or 4 times that written for
// each token and head.
#include "paged_internal.cuh"

namespace aqua {

namespace {

constexpr int D = kHeadDim;
constexpr int kThreads = 256;
constexpr int kTok = 128;                  // tokens per block

struct GatherParams {
  const int32_t* len;
  const int32_t* seq_idx;
  void* k;
  void* v;
  int32_t* dst_len;
  int32_t* n_abs;
  int Tcap, max_len;
};

// sixteen codes times s, stored as sixteen consecutive elements (the first n of them)
__device__ __forceinline__ void store16(float* p, const uint4& w, float s, int n) {
  const uint32_t* x = reinterpret_cast<const uint32_t*>(&w);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = e4m3x2_to_f32x2((uint16_t)(x[i] & 0xffffu)), b = e4m3x2_to_f32x2((uint16_t)(x[i] >> 16));
    const float4 f = make_float4(a.x * s, a.y * s, b.x * s, b.y * s);
    if (n >= 16) {
      reinterpret_cast<float4*>(p)[i] = f;
    } else {
      if (4 * i + 0 < n) p[4 * i + 0] = f.x;
      if (4 * i + 1 < n) p[4 * i + 1] = f.y;
      if (4 * i + 2 < n) p[4 * i + 2] = f.z;
      if (4 * i + 3 < n) p[4 * i + 3] = f.w;
    }
  }
}
__device__ __forceinline__ void store16(__nv_bfloat16* p, const uint4& w, float s, int n) {
  const uint32_t* x = reinterpret_cast<const uint32_t*>(&w);
  uint32_t y[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = e4m3x2_to_f32x2((uint16_t)(x[i] & 0xffffu)), b = e4m3x2_to_f32x2((uint16_t)(x[i] >> 16));
    y[2 * i] = pack_bf16(a.x * s, a.y * s);
    y[2 * i + 1] = pack_bf16(b.x * s, b.y * s);
  }
  if (n >= 16) {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(y[0], y[1], y[2], y[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(y[4], y[5], y[6], y[7]);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < n) reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)(y[i >> 1] >> (16 * (i & 1)));
  }
}

// One block per (128 tokens, head, destination sequence).
template <typename T>
__global__ void __launch_bounds__(kThreads) paged_gather_kernel(PagedView c, GatherParams g) {
  const int i = blockIdx.z, h = blockIdx.y, t0 = blockIdx.x * kTok;
  const int b = g.seq_idx ? __ldg(g.seq_idx + i) : i;
  bool bad = b < 0 || b >= c.B;
  const int n = bad ? 0 : checked_len(__ldg(g.len + b), c, g.max_len, bad);
  if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0) {
    if (bad) report_arg(c);
    g.dst_len[i] = n;
    if (g.n_abs) g.n_abs[i] = n;
  }
  if (t0 >= n) return;
  __shared__ int pids[kTok / 16];
  if (threadIdx.x < kTok / 16) {
    const int t = t0 + 16 * threadIdx.x;
    int pid = -1;
    if (t < n) {
      pid = __ldg(c.table + (size_t)b * c.max_pages + (t >> c.page_log2));
      if (pid < 0 || pid >= c.n_pages) {
        pid = -1;
        report_arg(c);
      }
    }
    pids[threadIdx.x] = pid;
  }
  __syncthreads();
  const int nt = min(kTok, n - t0), mask = (1 << c.page_log2) - 1;
  const size_t unit = (size_t)i * c.Hkv + h;
  T* kd = static_cast<T*>(g.k) + unit * c.m * (size_t)g.Tcap;
  T* vd = static_cast<T*>(g.v) + unit * (size_t)g.Tcap * D;
  for (int x = threadIdx.x; x < c.m * (kTok / 16); x += kThreads) {        // (dimension, 16 tokens)
    const int j = x >> 3, cc = x & 7, t = 16 * cc;
    if (t >= nt) continue;
    const int pid = pids[cc];
    uint4 w = make_uint4(0, 0, 0, 0);
    float s = 0.f;
    if (pid >= 0) {
      w = __ldg(reinterpret_cast<const uint4*>(c.k + c.kblock(pid, h) + ((size_t)j << c.page_log2) + ((t0 + t) & mask)));
      s = __ldg(c.ks + (size_t)pid * c.Hkv + h);
    }
    store16(kd + (size_t)j * g.Tcap + t0 + t, w, s, nt - t);
  }
  for (int x = threadIdx.x; x < nt * (D / 16); x += kThreads) {            // (token, 16 dimensions)
    const int t = x >> 3, cc = x & 7;
    const int pid = pids[t >> 4];
    uint4 w = make_uint4(0, 0, 0, 0);
    float s = 0.f;
    if (pid >= 0) {
      w = __ldg(reinterpret_cast<const uint4*>(c.v + c.vblock(pid, h) + (size_t)((t0 + t) & mask) * D) + cc);
      s = __ldg(c.vs + (size_t)pid * c.Hkv + h);
    }
    store16(vd + (size_t)(t0 + t) * D + 16 * cc, w, s, 16);
  }
}

}  // namespace

int launch_paged_gather(const PagedView& c, const int32_t* len, const int32_t* seq_idx, aqua_cache* dst, int max_len,
                        cudaStream_t st) {
  GatherParams g;
  g.len = len; g.seq_idx = seq_idx; g.k = dst->k_proj; g.v = dst->v; g.dst_len = dst->len; g.n_abs = dst->n_abs;
  g.Tcap = dst->Tcap; g.max_len = max_len;
  const dim3 grid((max_len + kTok - 1) / kTok > 0 ? (max_len + kTok - 1) / kTok : 1, c.Hkv, dst->B);
  if (dst->dtype == AQUA_BF16)
    paged_gather_kernel<__nv_bfloat16><<<grid, kThreads, 0, st>>>(c, g);
  else
    paged_gather_kernel<float><<<grid, kThreads, 0, st>>>(c, g);
  return check_launch("paged_gather_kernel");
}

}  // namespace aqua
