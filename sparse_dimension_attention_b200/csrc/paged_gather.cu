// Pages of the 8-bit cache back into a contiguous f32 or bf16 cache: every code
// times its page's scale, keys dimension-major, values token-major.
//
// A copy bound by memory: (m + 128) bytes read and 2 or 4 times that written for
// each token and head.  16 ragged sequences of up to 16384 tokens, 8 heads, to bf16:
// 122 us against 106 at the copy rate (87 %).
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

// Sixteen codes times s, stored as sixteen consecutive elements (the first n of them).  All lanes of a warp call it,
// neighbours with neighbouring destinations.
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
  // A lane has two 16-byte pieces.  Even and odd lanes trade one each, so that a store of the warp covers
  // pieces that lie side by side: first the even lanes' 32 bytes, then the odd lanes'.
  const bool odd = threadIdx.x & 1, pair = __all_sync(0xffffffffu, n >= 16);
  if (pair) {
    const uint64_t mine = reinterpret_cast<uint64_t>(p), other = __shfl_xor_sync(0xffffffffu, mine, 1);
    uint32_t got[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) got[i] = __shfl_xor_sync(0xffffffffu, odd ? y[i] : y[4 + i], 1);
    uint4* const e = reinterpret_cast<uint4*>(odd ? other : mine);           // the even lane's place
    uint4* const o = reinterpret_cast<uint4*>(odd ? mine : other);
    e[odd] = odd ? make_uint4(got[0], got[1], got[2], got[3]) : make_uint4(y[0], y[1], y[2], y[3]);
    o[odd] = odd ? make_uint4(y[4], y[5], y[6], y[7]) : make_uint4(got[0], got[1], got[2], got[3]);
  } else if (n >= 16) {
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
  __shared__ float scales[2][kTok / 16];
  if (threadIdx.x < kTok / 16) {
    const int t = t0 + 16 * threadIdx.x;
    int pid = -1;
    float ks = 0.f, vs = 0.f;
    if (t < n) {
      pid = __ldg(c.table + (size_t)b * c.max_pages + (t >> c.page_log2));
      if (pid >= 0 && pid < c.n_pages) {
        ks = __ldg(c.ks + (size_t)pid * c.Hkv + h);
        vs = __ldg(c.vs + (size_t)pid * c.Hkv + h);
      } else {
        pid = -1;
        report_arg(c);
      }
    }
    pids[threadIdx.x] = pid;
    scales[0][threadIdx.x] = ks;
    scales[1][threadIdx.x] = vs;
  }
  __syncthreads();
  const int nt = min(kTok, n - t0), mask = (1 << c.page_log2) - 1;
  const size_t unit = (size_t)i * c.Hkv + h;
  T* kd = static_cast<T*>(g.k) + unit * c.m * (size_t)g.Tcap + t0;
  T* vd = static_cast<T*>(g.v) + (unit * (size_t)g.Tcap + t0) * D;
  // A thread has piece cc of up to four dims (16 tokens each) and of up to four tokens (16 dims each): all eight
  // loads are in flight before the first store.
  constexpr int kEach = D * (kTok / 16) / kThreads;
  const int cc = threadIdx.x & 7, r0 = threadIdx.x >> 3, kpid = pids[cc];
  uint4 kw[kEach], vw[kEach];
#pragma unroll
  for (int y = 0; y < kEach; ++y) {
    const int j = r0 + y * (kThreads / 8);                     // dim, token
    kw[y] = vw[y] = make_uint4(0, 0, 0, 0);
    if (j < c.m && kpid >= 0)
      kw[y] = __ldg(reinterpret_cast<const uint4*>(c.k + c.kblock(kpid, h) + ((size_t)j << c.page_log2) + ((t0 + 16 * cc) & mask)));
    const int vpid = pids[j >> 4];
    if (j < nt && vpid >= 0)
      vw[y] = __ldg(reinterpret_cast<const uint4*>(c.v + c.vblock(vpid, h) + (size_t)((t0 + j) & mask) * D) + cc);
  }
#pragma unroll
  for (int y = 0; y < kEach; ++y) {
    const int j = r0 + y * (kThreads / 8);
    store16(kd + (size_t)j * g.Tcap + 16 * cc, kw[y], scales[0][cc], j < c.m ? nt - 16 * cc : 0);
  }
#pragma unroll
  for (int y = 0; y < kEach; ++y) {
    const int j = r0 + y * (kThreads / 8);
    store16(vd + (size_t)j * D + 16 * cc, vw[y], scales[1][j >> 4], j < nt ? 16 : 0);
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
