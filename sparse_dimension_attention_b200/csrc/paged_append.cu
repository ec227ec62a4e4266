// Append to the paged 8-bit cache: rotate, project, quantise, scatter.
//
// For every new token at slot t of its sequence and KV head g:
//   k~ = rope(k, t) P[g][:, :m]                       (f32)
//   s  = smallest power of two with max |x| <= 448 s over the values appended to the page,
//        or the page's own scale if that is larger and the page holds tokens already
//   code = e4m3(x / s);  the page's older codes are re-coded by s_old / s when s grew
// (edgentiq, "How AQUA Works", Online Inference: keys are projected before they are cached.)
#include "paged_internal.cuh"

namespace aqua {

namespace {

constexpr int D = kHeadDim;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kGroup = 8;                  // tokens projected per pass
constexpr int kRows = D / kWarps;          // input dims per warp

struct AppendParams {
  const void* k_new;
  const void* v_new;
  Strides ks, vs;
  const int32_t* start;
  const int32_t* cu;                       // nullptr: token b belongs to sequence b
  const float* P;
  RopeView rope;
  int n_tokens;
};

// A run of new tokens inside one page.
struct Segment {
  int b;          // sequence
  int token;      // first row of k_new / v_new
  int slot;       // first slot of the sequence
  int n;          // tokens, all in one page
};

// New tokens of sequence b (0, reported, where the device data do not allow them).
__device__ __forceinline__ int run_length(const AppendParams& a, const PagedView& c, int b, int& token, int& start,
                                          bool& bad) {
  start = __ldg(a.start + b);
  int n;
  if (a.cu == nullptr) {
    token = b;
    n = 1;
    bad = false;
  } else {
    token = __ldg(a.cu + b);
    const int end = __ldg(a.cu + b + 1);
    bad = token < 0 || end < token || end > a.n_tokens;
    n = bad ? 0 : end - token;
  }
  if (n > 0 && (start < 0 || (long long)start + n > c.capacity() ||
                (a.rope.cs != nullptr && (long long)start + n > a.rope.n_pos)))
    bad = true;
  return bad ? 0 : n;
}

// The segment with index `want` in the order of sequences and pages; false past the last one.
__device__ bool find_segment(const AppendParams& a, const PagedView& c, int want, Segment& s) {
  __shared__ int warp_sum[kWarps];
  __shared__ Segment found;
  __shared__ int have;
  if (threadIdx.x == 0) have = 0;
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int before = 0;
  for (int base = 0; base < c.B; base += kThreads) {
    const int b = base + threadIdx.x;
    int token = 0, start = 0, n = 0, pages = 0;
    if (b < c.B) {
      bool bad;
      n = run_length(a, c, b, token, start, bad);
      if (bad && want == 0) report_arg(c);
      if (n > 0) pages = ((start + n - 1) >> c.page_log2) - (start >> c.page_log2) + 1;
    }
    int sum = pages;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    __syncthreads();                       // warp_sum free again, have initialised
    if (lane == 31) warp_sum[w] = sum;
    __syncthreads();
    int off = before, total = 0;
    for (int x = 0; x < kWarps; ++x) {
      if (x < w) off += warp_sum[x];
      total += warp_sum[x];
    }
    const int first = off + sum - pages;
    if (pages > 0 && want >= first && want < first + pages) {
      const int page0 = (start >> c.page_log2) + (want - first);
      const int lo = max(start, page0 << c.page_log2), hi = min(start + n, (page0 + 1) << c.page_log2);
      found.b = b;
      found.token = token + (lo - start);
      found.slot = lo;
      found.n = hi - lo;
      have = 1;
    }
    before += total;
    __syncthreads();
    if (have) {
      s = found;
      if (want != 0) return true;          // segment 0's block also looks at every later sequence
    }
  }
  return have != 0;
}

template <typename T>
__device__ __forceinline__ void load4(const T* p, float (&f)[4]);
template <>
__device__ __forceinline__ void load4(const float* p, float (&f)[4]) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
}
template <>
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float (&f)[4]) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  f[0] = bf16lo(w.x); f[1] = bf16hi(w.x); f[2] = bf16lo(w.y); f[3] = bf16hi(w.y);
}

// four codes times ratio, nearest even; bytes whose bit in `keep` is clear stay as they are
__device__ __forceinline__ uint32_t recode4(uint32_t w, float ratio, uint32_t byte_mask) {
  const float2 a = e4m3x2_to_f32x2((uint16_t)(w & 0xffffu)), b = e4m3x2_to_f32x2((uint16_t)(w >> 16));
  const uint32_t r = f32x4_to_e4m3x4(a.x * ratio, a.y * ratio, b.x * ratio, b.y * ratio);
  return (r & byte_mask) | (w & ~byte_mask);
}

// Re-codes slots 0 .. fill-1 of a key block ([m][page] bytes) or a value block ([page][D]).
__device__ void recode_keys(uint8_t* blk, int m, int page_log2, int fill, float ratio, int tid, int nthreads) {
  const int page = 1 << page_log2, chunks = (m << page_log2) >> 4;
  for (int c = tid; c < chunks; c += nthreads) {
    const int s0 = (c << 4) & (page - 1);
    if (s0 >= fill) continue;
    uint4* p = reinterpret_cast<uint4*>(blk) + c;
    uint4 w = *p;
    uint32_t* x = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int left = fill - (s0 + 4 * i);            // slots of this word that hold tokens
      const uint32_t mask = left >= 4 ? 0xffffffffu : (left <= 0 ? 0u : (1u << (8 * left)) - 1u);
      x[i] = recode4(x[i], ratio, mask);
    }
    *p = w;
  }
}
__device__ void recode_values(uint8_t* blk, int fill, float ratio, int tid, int nthreads) {
  for (int c = tid; c < fill * (D / 16); c += nthreads) {
    uint4* p = reinterpret_cast<uint4*>(blk) + c;
    uint4 w = *p;
    uint32_t* x = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = recode4(x[i], ratio, 0xffffffffu);
    *p = w;
  }
}

// Scale of a page that takes values up to amax; fill: tokens it holds already.
__device__ __forceinline__ float page_scale(float amax, float old, int fill) {
  const float s = pow2_scale(amax);
  return fill > 0 ? fmaxf(old, s) : s;
}

// One block per (page segment, KV head).  A thread holds 16 rows x 4 columns of P
// in registers for the whole segment, so P is read once; eight tokens at a time
// are projected (warp w sums input dims 16w .. 16w+15) and their eight partial
// sums added in order.
template <typename T>
__global__ void __launch_bounds__(kThreads) paged_append_run_kernel(PagedView c, AppendParams a) {
  extern __shared__ __align__(16) float dyn[];
  float* kt = dyn;                                         // [page][D] projected keys
  float* part = kt + ((size_t)D << c.page_log2);           // [kWarps][kGroup][D]
  float* xs = part + kWarps * kGroup * D;                  // [kGroup][D] raw, then rotated rows
  float* raw = xs + kGroup * D;
  __shared__ float red[2][kWarps];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, h = blockIdx.y;
  Segment s;
  if (!find_segment(a, c, blockIdx.x, s)) return;
  const int pid = __ldg(c.table + (size_t)s.b * c.max_pages + (s.slot >> c.page_log2));
  if (pid < 0 || pid >= c.n_pages) {
    if (threadIdx.x == 0) report_arg(c);
    return;
  }
  const T* kr = static_cast<const T*>(a.k_new) + (size_t)s.token * a.ks.row + (size_t)h * a.ks.head;
  const T* vr = static_cast<const T*>(a.v_new) + (size_t)s.token * a.vs.row + (size_t)h * a.vs.head;
  float4 p[kRows];
  const float4* Pg = reinterpret_cast<const float4*>(a.P + (size_t)h * D * D);
#pragma unroll
  for (int i = 0; i < kRows; ++i) p[i] = __ldg(Pg + (w * kRows + i) * (D / 4) + lane);

  float kmax = 0.f, vmax = 0.f;
  for (int t0 = 0; t0 < s.n; t0 += kGroup) {
    const int nt = min(kGroup, s.n - t0);
    if (w < nt) {
      float f[4];
      load4<T>(kr + (size_t)(t0 + w) * a.ks.row + 4 * lane, f);
      *reinterpret_cast<float4*>(raw + w * D + 4 * lane) = make_float4(f[0], f[1], f[2], f[3]);
      __syncwarp();
      if (a.rope.cs != nullptr) {
        const float* cs = a.rope.cs + (size_t)(s.slot + t0 + w) * a.rope.rot;
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = rotated<float>(raw + w * D, 4 * lane + e, cs, a.rope.rot, a.rope.interleaved);
      }
      *reinterpret_cast<float4*>(xs + w * D + 4 * lane) = make_float4(f[0], f[1], f[2], f[3]);
      load4<T>(vr + (size_t)(t0 + w) * a.vs.row + 4 * lane, f);
#pragma unroll
      for (int e = 0; e < 4; ++e) vmax = fmaxf(vmax, finite_abs(f[e]));
    }
    __syncthreads();
    for (int t = 0; t < nt; ++t) {
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const float x = xs[t * D + w * kRows + i];
        acc.x = fmaf(x, p[i].x, acc.x); acc.y = fmaf(x, p[i].y, acc.y);
        acc.z = fmaf(x, p[i].z, acc.z); acc.w = fmaf(x, p[i].w, acc.w);
      }
      *reinterpret_cast<float4*>(part + (w * kGroup + t) * D + 4 * lane) = acc;
    }
    __syncthreads();
    if (w < nt) {
      float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int x = 0; x < kWarps; ++x) {
        const float4 q = *reinterpret_cast<const float4*>(part + (x * kGroup + w) * D + 4 * lane);
        y[0] += q.x; y[1] += q.y; y[2] += q.z; y[3] += q.w;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (4 * lane + e < c.m) kmax = fmaxf(kmax, finite_abs(y[e]));
      *reinterpret_cast<float4*>(kt + (size_t)(t0 + w) * D + 4 * lane) = make_float4(y[0], y[1], y[2], y[3]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    kmax = fmaxf(kmax, __shfl_xor_sync(0xffffffffu, kmax, o));
    vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, o));
  }
  if (lane == 0) {
    red[0][w] = kmax;
    red[1][w] = vmax;
  }
  __syncthreads();
  for (int x = 0; x < kWarps; ++x) {
    kmax = fmaxf(kmax, red[0][x]);
    vmax = fmaxf(vmax, red[1][x]);
  }
  const int fill = s.slot & ((1 << c.page_log2) - 1);
  const size_t si = (size_t)pid * c.Hkv + h;
  const float kold = c.ks[si], vold = c.vs[si];
  const float ks = page_scale(kmax, kold, fill), vs = page_scale(vmax, vold, fill);
  uint8_t* kb = c.k + c.kblock(pid, h);
  uint8_t* vb = c.v + c.vblock(pid, h);
  if (fill > 0 && ks != kold) recode_keys(kb, c.m, c.page_log2, fill, kold / ks, threadIdx.x, kThreads);
  if (fill > 0 && vs != vold) recode_values(vb, fill, vold / vs, threadIdx.x, kThreads);
  __syncthreads();                         // everybody has read the old scales; old codes are in place
  if (threadIdx.x == 0) {
    c.ks[si] = ks;
    c.vs[si] = vs;
  }
  const float ki = 1.f / ks, vi = 1.f / vs;
  // keys: one byte per (dimension, slot), consecutive threads on consecutive slots
  for (int i = threadIdx.x; i < c.m * s.n; i += kThreads) {
    const int j = i / s.n, t = i - j * s.n;
    kb[((size_t)j << c.page_log2) + fill + t] = (uint8_t)f32x2_to_e4m3x2(kt[(size_t)t * D + j] * ki, 0.f);
  }
  for (int t = w; t < s.n; t += kWarps) {
    float f[4];
    load4<T>(vr + (size_t)t * a.vs.row + 4 * lane, f);
    reinterpret_cast<uint32_t*>(vb + (size_t)(fill + t) * D)[lane] =
        f32x4_to_e4m3x4(f[0] * vi, f[1] * vi, f[2] * vi, f[3] * vi);
  }
}

// One new token for each sequence: a block takes up to kStepGroup sequences of one
// KV head.  Bound by latency: P (64 KB, from L2) is read once per block into
// registers before the wait on the previous kernel, and kept there as f64, whose
// 64 multiply-adds a cycle and SM are enough here; the sums are then exact to f32
// rounding, so that a code differs from the exact one only on a tie.  Warp t
// writes token t.
constexpr int kStepThreads = 512;
constexpr int kStepGroup = 16;
constexpr int kStepSlices = kStepThreads / D;              // slices of 32 input dims

template <typename T>
__global__ void __launch_bounds__(kStepThreads) paged_append_step_kernel(PagedView c, AppendParams a, int group) {
  extern __shared__ __align__(16) double part[];           // [kStepSlices][group][D]
  __shared__ __align__(16) double xs[kStepGroup][D];       // rotated rows
  __shared__ float raw[kStepGroup][D];
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, h = blockIdx.y;
  const int col = tid & (D - 1), sl = tid >> 7;
  constexpr int R = D / kStepSlices;
  float pf[R];
  {
    const float* Pg = a.P + ((size_t)h * D + sl * R) * D + col;
#pragma unroll
    for (int i = 0; i < R; ++i) pf[i] = __ldg(Pg + (size_t)i * D);
  }
  pdl_wait();
  const int b = blockIdx.x * group + w, nt = min(group, c.B - (int)blockIdx.x * group);
  int pid = -1, slot = 0;
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  if (w < nt) {
    int token, n;
    bool bad;
    n = run_length(a, c, b, token, slot, bad);
    if (n > 0) {
      pid = __ldg(c.table + (size_t)b * c.max_pages + (slot >> c.page_log2));
      if (pid < 0 || pid >= c.n_pages) {
        pid = -1;
        bad = true;
      }
    }
    if (bad && lane == 0) report_arg(c);
    if (pid >= 0) {
      float f[4];
      load4<T>(static_cast<const T*>(a.k_new) + (size_t)token * a.ks.row + (size_t)h * a.ks.head + 4 * lane, f);
      load4<T>(static_cast<const T*>(a.v_new) + (size_t)token * a.vs.row + (size_t)h * a.vs.head + 4 * lane, v);
      *reinterpret_cast<float4*>(&raw[w][4 * lane]) = make_float4(f[0], f[1], f[2], f[3]);
      __syncwarp();
      const float* cs = a.rope.cs + (size_t)slot * a.rope.rot;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        xs[w][4 * lane + e] =
            a.rope.cs != nullptr ? rotated<double>(raw[w], 4 * lane + e, cs, a.rope.rot, a.rope.interleaved) : (double)f[e];
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) xs[w][4 * lane + e] = 0.0;
    }
  }
  double p[R];
#pragma unroll
  for (int i = 0; i < R; ++i) p[i] = pf[i];
  __syncthreads();
  for (int t = 0; t < nt; ++t) {
    double s0 = 0.0, s1 = 0.0;
#pragma unroll
    for (int i = 0; i < R; i += 2) {
      const double2 x = *reinterpret_cast<const double2*>(&xs[t][sl * R + i]);
      s0 = fma(x.x, p[i], s0);
      s1 = fma(x.y, p[i + 1], s1);
    }
    part[(sl * group + t) * D + col] = s0 + s1;
  }
  __syncthreads();
  if (pid < 0) return;
  float y[4];
  float kmax = 0.f, vmax = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const double* q = part + w * D + lane + 32 * e;        // lane's dims: lane + 32 e
    double sum = q[0];
#pragma unroll
    for (int x = 1; x < kStepSlices; ++x) sum += q[(size_t)x * group * D];
    y[e] = (float)sum;
    if (lane + 32 * e < c.m) kmax = fmaxf(kmax, finite_abs(y[e]));
    vmax = fmaxf(vmax, finite_abs(v[e]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    kmax = fmaxf(kmax, __shfl_xor_sync(0xffffffffu, kmax, o));
    vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, o));
  }
  const int fill = slot & ((1 << c.page_log2) - 1);
  const size_t si = (size_t)pid * c.Hkv + h;
  const float kold = fill > 0 ? c.ks[si] : 0.f, vold = fill > 0 ? c.vs[si] : 0.f;
  const float ks = page_scale(kmax, kold, fill), vs = page_scale(vmax, vold, fill);
  uint8_t* kb = c.k + c.kblock(pid, h);
  uint8_t* vb = c.v + c.vblock(pid, h);
  if (fill > 0 && ks != kold) recode_keys(kb, c.m, c.page_log2, fill, kold / ks, lane, 32);
  if (fill > 0 && vs != vold) recode_values(vb, fill, vold / vs, lane, 32);
  __syncwarp();                            // a 16-byte piece re-coded by one lane holds another lane's new byte
  if (lane == 0) {
    c.ks[si] = ks;
    c.vs[si] = vs;
  }
  const float ki = 1.f / ks, vi = 1.f / vs;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int j = lane + 32 * e;
    if (j < c.m) kb[((size_t)j << c.page_log2) + fill] = (uint8_t)f32x2_to_e4m3x2(y[e] * ki, 0.f);
  }
  reinterpret_cast<uint32_t*>(vb + (size_t)fill * D)[lane] =
      f32x4_to_e4m3x4(v[0] * vi, v[1] * vi, v[2] * vi, v[3] * vi);
}

template <typename T>
int launch_step(const PagedView& c, const AppendParams& a, cudaStream_t st) {
  // enough sequences a block that the blocks fit the SMs at once
  const int want = (c.B * c.Hkv + device_sm_count() - 1) / device_sm_count();
  const int group = want < kStepGroup ? want : kStepGroup;
  const int smem = kStepSlices * group * D * (int)sizeof(double);
  const int rc = set_smem_limit(paged_append_step_kernel<T>, kStepSlices * kStepGroup * D * (int)sizeof(double),
                                "paged_append_step_kernel");
  if (rc != AQUA_OK) return rc;
  const cudaError_t e = launch_pdl(paged_append_step_kernel<T>, dim3((c.B + group - 1) / group, c.Hkv),
                                   dim3(kStepThreads), smem, st, c, a, group);
  if (e != cudaSuccess) return set_error(AQUA_ERR_CUDA, "paged_append_step_kernel: %s", cudaGetErrorString(e));
  return check_launch("paged_append_step_kernel");
}

template <typename T>
int launch_run(const PagedView& c, const AppendParams& a, cudaStream_t st) {
  const int smem = ((D << c.page_log2) + kWarps * kGroup * D + 2 * kGroup * D) * (int)sizeof(float);
  const int rc = set_smem_limit(paged_append_run_kernel<T>, smem, "paged_append_run_kernel");
  if (rc != AQUA_OK) return rc;
  // a run of n >= 1 tokens touches at most (n - 2) / page + 2 pages, and at most n
  const long long by_page = a.n_tokens / (1 << c.page_log2) + 2LL * c.B;
  const unsigned segs = (unsigned)(by_page < a.n_tokens ? by_page : a.n_tokens);
  paged_append_run_kernel<T><<<dim3(segs, c.Hkv), kThreads, smem, st>>>(c, a);
  return check_launch("paged_append_run_kernel");
}

}  // namespace

int launch_paged_append(const PagedView& c, const void* k_new, const void* v_new, bool bf16, const Strides& ks,
                        const Strides& vs, int n_tokens, const int32_t* start, const int32_t* cu, const float* P,
                        const RopeView& rope, cudaStream_t st) {
  AppendParams a;
  a.k_new = k_new; a.v_new = v_new; a.ks = ks; a.vs = vs; a.start = start; a.cu = cu;
  a.P = P; a.rope = rope; a.n_tokens = n_tokens;
  if (cu == nullptr) return bf16 ? launch_step<__nv_bfloat16>(c, a, st) : launch_step<float>(c, a, st);
  return bf16 ? launch_run<__nv_bfloat16>(c, a, st) : launch_run<float>(c, a, st);
}

}  // namespace aqua
