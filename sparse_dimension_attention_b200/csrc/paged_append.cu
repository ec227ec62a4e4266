// Append to the paged 8-bit cache: rotate, project, quantise, scatter.
//
// For every new token at slot t of its sequence and KV head g:
//   k~ = rope(k, t) P[g][:, :m]                       (f64, f32 or two f16 parts of each factor: see the kernels)
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

// four codes times ratio, nearest even; bytes that byte_mask leaves out stay as they are
__device__ __forceinline__ uint32_t recode4(uint32_t w, float ratio, uint32_t byte_mask) {
  const float2 a = e4m3x2_to_f32x2((uint16_t)(w & 0xffffu)), b = e4m3x2_to_f32x2((uint16_t)(w >> 16));
  const uint32_t r = f32x4_to_e4m3x4(a.x * ratio, a.y * ratio, b.x * ratio, b.y * ratio);
  return (r & byte_mask) | (w & ~byte_mask);
}

// Re-codes slots 0 .. fill-1 of a key block ([m][page] bytes) or a value block ([page][D]).  Rare: kept out of
// the kernels' loops.
__device__ __noinline__ void recode_keys(uint8_t* blk, int m, int page_log2, int fill, float ratio, int tid, int nthreads) {
  const int page = 1 << page_log2, chunks = (m << page_log2) >> 4;
#pragma unroll 1
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
__device__ __noinline__ void recode_values(uint8_t* blk, int fill, float ratio, int tid, int nthreads) {
#pragma unroll 1
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

// Rows are rotated and summed times 2^-16 (unless they are brought to one size anyway), so that a sum of large numbers
// is an infinity only where the result is one; exact for all above 2^-110, and what is smaller has the code 0.
constexpr float kDown = 1.f / 65536.f;

// A block takes page segments of one KV head.  A thread holds 16 rows x 4 columns of
// P in registers, so P is read once; eight tokens at a time are projected (warp w
// sums input dims 16w .. 16w+15) and their eight partial sums added in order.
// Bound by the reads of the rows from shared memory, 0.3 us a token and block.
template <typename T>
__global__ void __launch_bounds__(kThreads) paged_append_run_kernel(PagedView c, AppendParams a) {
  extern __shared__ __align__(16) float dyn[];
  float* kt = dyn;                                         // [page][D] projected keys
  float* part = kt + ((size_t)D << c.page_log2);           // [kWarps][kGroup][D]
  float* xs = part + kWarps * kGroup * D;                  // [kGroup][D] raw, then rotated rows
  float* raw = xs + kGroup * D;
  __shared__ float red[2][kWarps];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, h = blockIdx.y;
  float4 p[kRows];
  const float4* Pg = reinterpret_cast<const float4*>(a.P + (size_t)h * D * D);
#pragma unroll
  for (int i = 0; i < kRows; ++i) p[i] = __ldg(Pg + (w * kRows + i) * (D / 4) + lane);
#pragma unroll 1
  for (int seg = blockIdx.x;; seg += gridDim.x) {          // to the last segment the device data give
    __syncthreads();                         // the search's shared words are free again
    Segment s;
    if (!find_segment(a, c, seg, s)) return;
    const int pid = __ldg(c.table + (size_t)s.b * c.max_pages + (s.slot >> c.page_log2));
    if (pid < 0 || pid >= c.n_pages) {
      if (threadIdx.x == 0) report_arg(c);
      continue;
    }
    const T* kr = static_cast<const T*>(a.k_new) + (size_t)s.token * a.ks.row + (size_t)h * a.ks.head;
    const T* vr = static_cast<const T*>(a.v_new) + (size_t)s.token * a.vs.row + (size_t)h * a.vs.head;

    float kmax = 0.f, vmax = 0.f;
    for (int t0 = 0; t0 < s.n; t0 += kGroup) {
      const int nt = min(kGroup, s.n - t0);
      if (w < nt) {
        float f[4];
        load4<T>(kr + (size_t)(t0 + w) * a.ks.row + 4 * lane, f);
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] *= kDown;
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
        for (int e = 0; e < 4; ++e) {
          y[e] *= 1.f / kDown;
          if (4 * lane + e < c.m) kmax = fmaxf(kmax, finite_abs(y[e]));
        }
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
}

// ------------------------------------------------------------------ runs of tokens on the tensor cores
//
// A tile is 128 slots of a sequence, aligned, so whole pages; persistent blocks,
// one an SM, each of one head, share the tiles.  k~ = x P on tcgen05 with
// both factors split into two f16 parts (x_l P_l + x_l P_h + x_h P_l + x_h P_h, f32
// accumulation): rows and P are first brought to [2^10, 2^11) by powers of two,
// so the parts hold 22 bits.  The tensor cores cut every sum they extend off to 24
// bits, which makes one chain of a row's products 2.3e-7 off (2-norm; an f32 sum of
// 128 terms 2.0e-7).  So two accumulators of 64 input dims each, the small products
// first, added in f32: of 40 calls of 701 f32 tokens and 4 heads 70 codes fall on
// the other side of a tie (92 without x_l P_l, which costs 1 %; 115 with the rows
// projected by a library's f32 product).
//
// What bounds it is the arithmetic around the products (some 20 instructions an
// element), so the roles overlap: warps 0-7 rotate, normalise and split the rows
// of a tile, warps 8-11 turn projected rows into codes, warps 12-19 do the
// values, one lane issues the products.  Operands and accumulators are double.
// The loops are kept short (rolled over 32 rows or 32 columns): unrolled, the
// roles together were 122 KB of code and mostly waited for instructions.
// Measured: 8 ragged prompts of 16384 tokens together, 8 heads: bf16 64 us (the
// bytes alone: 17), f32 72 us (27); 5.5 us a tile and SM, most of it the row warps'.
constexpr int kTile = 128;
constexpr int kRowThreads = 256, kKeyThreads = 128, kValThreads = 256;
constexpr int kKeyWarp0 = kRowThreads / 32, kValWarp0 = kKeyWarp0 + kKeyThreads / 32;
constexpr int kProdWarp = kValWarp0 + kValThreads / 32;
constexpr int kTileThreads = (kProdWarp + 1) * 32;
constexpr int kGroups = kTile / 16;        // groups of 16 slots
constexpr int kPart = kTile * D * 2;       // bytes of one f16 part of a 128 x 128 operand
enum NamedBar { kBarKey = 1, kBarVal = 2, kBarRow = 3 };

// tiles (128-slot blocks) that a run of n tokens from slot `start` touches
__device__ __forceinline__ int run_tiles(int start, int n) { return n > 0 ? ((start + n - 1) >> 7) - (start >> 7) + 1 : 0; }

// Tile ti of the run of sequence b.
struct Walk {
  int b, start, token, n, ti;
  __device__ __forceinline__ int base() const { return ((start >> 7) + ti) << 7; }          // first slot of the tile
  __device__ __forceinline__ int lo() const { return max(start, base()) - base(); }          // new slots of the tile
  __device__ __forceinline__ int hi() const { return min(start + n, base() + kTile) - base(); }
  __device__ __forceinline__ void next(const PagedView& c, const AppendParams& a) {         // there is one
    if (++ti < run_tiles(start, n)) return;
    ti = 0;
    do {
      bool bad;
      n = run_length(a, c, ++b, token, start, bad);
    } while (n == 0);
  }
  // tokens that the page of slot group g held before: the page the run starts in, when it starts inside
  __device__ __forceinline__ int held(const PagedView& c, int g) const {
    return ti == 0 && (base() + 16 * g) >> c.page_log2 == start >> c.page_log2 ? start & ((1 << c.page_log2) - 1) : 0;
  }
  // page of slot group g if the run has tokens in it (-1: none, or no such page)
  __device__ __forceinline__ int page_of(const PagedView& c, int g) const {
    if (16 * g >= hi() || 16 * g + 16 <= lo()) return -1;
    const int pid = __ldg(c.table + (size_t)b * c.max_pages + ((base() + 16 * g) >> c.page_log2));
    if (pid >= 0 && pid < c.n_pages) return pid;
    report_arg(c);
    return -1;
  }
};

struct TileMisc {
  uint64_t x_full[2], x_free[2], d_full[2], d_free[2];
  float unit[4][kTile];                    // power of two that undoes a row's and P's normalisation
  float kgroup[2][kGroups];                // largest magnitude of every 16 slots, of even and odd tiles
  float vgroup[kValThreads / 32][kGroups];
  float vinv[kGroups];                     // 1 / scale of every 16 slots' page
  int vpid[kGroups];                       // their page, -1: none
  float vrecode;                           // factor for the codes an open page holds already (1: none)
  uint32_t pmax;
  uint32_t tmem;
  int scan[kTileThreads / 32];
  Walk at;                                 // the block's first tile
  int abort;
};

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// two floats as a packed pair of f16, and what the pair leaves
__device__ __forceinline__ uint32_t split_pair(float& x0, float& x1) {
  const uint32_t h = pack_half2(x0, x1);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  x0 -= f.x;
  x1 -= f.y;
  return h;
}

// byte offset of eight columns from `col` (a multiple of 8) of a row in a part: two halves of 64 columns, rows
// of 128 bytes, 128-byte swizzle
__device__ __forceinline__ uint32_t part_off(int row, int col) {
  return (uint32_t)((col >> 6) * (kTile * 128) + row * 128 + ((((col & 63) >> 3) ^ (row & 7)) << 4));
}

__device__ __forceinline__ uint64_t desc_sw128(uint32_t addr, uint32_t lbo) {
  return (uint64_t)((addr >> 4) & 0x3FFF) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ void mma_f16(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}
__device__ __forceinline__ void commit_to(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// 32 columns of this warp's lanes; the registers hold them after tmem_wait_ld
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&a)[32], uint32_t (&b)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(a[i]), "+r"(b[i]));      // not before the wait
}

// power of two that brings a largest magnitude f * 2^e to [2^10, 2^11), and its inverse
__device__ __forceinline__ float norm_up(float mx, float& undo) {
  const int e = min(max((int)(__float_as_uint(mx) >> 23) - 127, -100), 127);
  undo = __uint_as_float((uint32_t)(e - 10 + 127) << 23);
  return __uint_as_float((uint32_t)(10 - e + 127) << 23);
}

// eight consecutive elements as f32
__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  const float4 u = __ldg(reinterpret_cast<const float4*>(p)), v = __ldg(reinterpret_cast<const float4*>(p) + 1);
  f[0] = u.x; f[1] = u.y; f[2] = u.z; f[3] = u.w; f[4] = v.x; f[5] = v.y; f[6] = v.z; f[7] = v.w;
}
// the same eight elements, as they lie
template <typename T> struct Raw8;
template <> struct Raw8<float> {
  float4 u, v;
  __device__ __forceinline__ void load(const float* p) {
    u = __ldg(reinterpret_cast<const float4*>(p));
    v = __ldg(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void get(float* f) const {
    f[0] = u.x; f[1] = u.y; f[2] = u.z; f[3] = u.w; f[4] = v.x; f[5] = v.y; f[6] = v.z; f[7] = v.w;
  }
  // times a power of two
  __device__ __forceinline__ void scale(float p) {
    u = make_float4(u.x * p, u.y * p, u.z * p, u.w * p);
    v = make_float4(v.x * p, v.y * p, v.z * p, v.w * p);
  }
  // largest magnitude, NaN passed over
  __device__ __forceinline__ float amax() const {
    return fmaxf(fmaxf(fmaxf(fabsf(u.x), fabsf(u.y)), fmaxf(fabsf(u.z), fabsf(u.w))),
                 fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))));
  }
};
template <> struct Raw8<__nv_bfloat16> {
  uint4 w;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { w = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void get(float* f) const {
    f[0] = bf16lo(w.x); f[1] = bf16hi(w.x); f[2] = bf16lo(w.y); f[3] = bf16hi(w.y);
    f[4] = bf16lo(w.z); f[5] = bf16hi(w.z); f[6] = bf16lo(w.w); f[7] = bf16hi(w.w);
  }
  __device__ __forceinline__ void scale(float f) {
    const __nv_bfloat162 s = __float2bfloat162_rn(f);
    __nv_bfloat162* p = reinterpret_cast<__nv_bfloat162*>(&w);
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = __hmul2(p[i], s);
  }
  __device__ __forceinline__ float amax() const {
    const __nv_bfloat162* p = reinterpret_cast<const __nv_bfloat162*>(&w);
    const __nv_bfloat162 m = __hmax2(__hmax2(__habs2(p[0]), __habs2(p[1])), __hmax2(__habs2(p[2]), __habs2(p[3])));
    return fmaxf(__bfloat162float(m.x), __bfloat162float(m.y));
  }
};

// largest finite magnitude of eight elements: the path of rows with an infinity, kept out of the loops
template <typename T>
__device__ __noinline__ float finite_amax8(const T* p) {
  float m = 0.f;
  for (int e = 0; e < 8; ++e) m = fmaxf(m, finite_abs(Elem<T>::load(p + e)));
  return m;
}

// Bounded wait; after a time-out every later wait returns at once and the roles run through their loops (all
// named barriers are met), writing garbage in bounds.
__device__ __forceinline__ void tile_wait(uint64_t* bar, uint32_t parity, TileMisc& ms, int32_t* ctrl) {
  if (!mbar_try_wait(bar, parity) && !*(volatile int*)&ms.abort && !mbar_wait_bounded(bar, parity)) {
    *(volatile int*)&ms.abort = 1;
    record_status(ctrl, AQUA_ERR_TIMEOUT);
  }
  __syncwarp();
}

// How a row is rotated: pairs (i, i + rot / 2) or (2 i, 2 i + 1) in blocks of eight (rot a multiple of 16, or no
// rotation), or dim by dim.  One kernel for each: three roles' loops share the instruction cache, and a
// kernel that held all three forms waited for instructions most of the time.
enum RotMode { kHalves = 0, kPairs = 1, kAnyRot = 2 };

template <typename T, int MODE>
__global__ void __launch_bounds__(kTileThreads, 1) paged_append_tile_kernel(PagedView c, AppendParams a) {
  extern __shared__ __align__(1024) uint8_t tile_smem[];
  uint8_t* const sP = tile_smem;                         // P: two f16 parts
  uint8_t* const sX = sP + 2 * kPart;                    // rows: two f16 parts, two buffers
  uint8_t* const sC = sX + 4 * kPart;                    // codes of a tile's keys, as its pages hold them; two buffers
  TileMisc& ms = *reinterpret_cast<TileMisc*>(sC + 2 * D * kTile);
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, h = blockIdx.y;

  if (tid == 0) {
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ms.x_full[i], kRowThreads);
      mbar_init(&ms.x_free[i], 1);
      mbar_init(&ms.d_full[i], 1);
      mbar_init(&ms.d_free[i], kKeyThreads);
    }
    fence_barrier_init();
    ms.abort = 0;
    ms.pmax = 0;
  }
  if (w == kProdWarp) {
    // two accumulators of 128 columns for each of two tiles
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&ms.tmem)), "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  }
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = ms.tmem;
  prefetch_head(a.P + (size_t)h * D * D, tid, kTileThreads);
  pdl_wait();
  // ---- P of the head, normalised and split
  float p_undo;
  {
    constexpr int kEach = (D * D / 8 + kTileThreads - 1) / kTileThreads;
    Raw8<float> f[kEach];
    float mx = 0.f;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int e = tid + i * kTileThreads;
      if (e < D * D / 8) f[i].load(a.P + (size_t)h * D * D + 8 * e);
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i)
      if (tid + i * kTileThreads < D * D / 8) mx = fmaxf(mx, f[i].amax());
    mx = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mx)));
    if (lane == 0) atomicMax(&ms.pmax, __float_as_uint(mx));
    __syncthreads();
    const float up = norm_up(__uint_as_float(ms.pmax), p_undo);
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int e = tid + i * kTileThreads, row = e >> 4, col = (e & 15) * 8;
      if (e >= D * D / 8) break;
      float x[8];
      f[i].scale(up);
      f[i].get(x);
      uint32_t hw[4], lw[4];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        // columns past d_store are not stored: zeros, so that they set no maximum
        float x0 = col + 2 * y < c.m ? x[2 * y] : 0.f, x1 = col + 2 * y + 1 < c.m ? x[2 * y + 1] : 0.f;
        hw[y] = split_pair(x0, x1);
        lw[y] = pack_half2(x0, x1);
      }
      *reinterpret_cast<uint4*>(sP + part_off(row, col)) = make_uint4(hw[0], hw[1], hw[2], hw[3]);
      *reinterpret_cast<uint4*>(sP + kPart + part_off(row, col)) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
    }
    fence_proxy_async_smem();
  }

  // ---- this block's share of the tiles: exclusive sums of the runs' tiles, a pass per kTileThreads sequences
  int n_tiles = 0, i0 = 0, n_my = 0;
  Walk at = {0, 0, 0, 0, 0};
  const bool once = c.B <= kTileThreads;     // one pass finds the total and, from the same registers, the first tile
#pragma unroll 1
  for (int round = 0; round < (once ? 1 : 2); ++round) {
    int before = 0;
#pragma unroll 1
    for (int base = 0; base < c.B; base += kTileThreads) {
      Walk mine = {base + tid, 0, 0, 0, 0};
      int x = 0;
      if (mine.b < c.B) {
        bool bad;
        mine.n = run_length(a, c, mine.b, mine.token, mine.start, bad);
        if (bad && blockIdx.x == 0 && round == 0) report_arg(c);
        x = run_tiles(mine.start, mine.n);
      }
      int sum = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += y;
      }
      __syncthreads();
      if (lane == 31) ms.scan[w] = sum;
      __syncthreads();
      int off = before, all = 0;
#pragma unroll
      for (int y = 0; y < kTileThreads / 32; ++y) {
        if (y < w) off += ms.scan[y];
        all += ms.scan[y];
      }
      before += all;
      if (once) n_tiles = all;
      if (once || round == 1) {
        i0 = (int)((long long)blockIdx.x * n_tiles / gridDim.x);
        n_my = (int)((long long)(blockIdx.x + 1) * n_tiles / gridDim.x) - i0;
        if (x > 0 && i0 >= off + sum - x && i0 < off + sum) {
          mine.ti = i0 - (off + sum - x);
          ms.at = mine;
        }
      }
    }
    if (!once && round == 0) n_tiles = before;
  }
  __syncthreads();
  if (n_my > 0) at = ms.at;

  if (w < kKeyWarp0) {
    // ================= rows: rotate, normalise, split =================
    // eight lanes a row, sixteen dims each: a block of eight rotated pairs, or sixteen dims past the rotation
    const int j8 = tid & 7, rot = a.rope.cs ? a.rope.rot : 0, half = rot >> 1;
    const bool turned = 8 * j8 < half, mixed = MODE != kHalves || !turned;
    const int da = mixed ? 16 * j8 : 8 * j8, db = mixed ? 16 * j8 + 8 : half + 8 * j8;
    Raw8<T> ra, rb;                                           // one pass ahead
    Walk ahead = at;
    int ahead_t = 0, ahead_pass = 0;
    auto fetch = [&]() {
      if (ahead_t < n_my) {
        const int r = (tid >> 3) + 32 * ahead_pass;
        if (r >= ahead.lo() && r < ahead.hi()) {
          const T* src = static_cast<const T*>(a.k_new) + (size_t)(ahead.token + ahead.base() + r - ahead.start) * a.ks.row +
                         (size_t)h * a.ks.head;
          ra.load(src + da);
          rb.load(src + db);
        }
        if (++ahead_pass == 4) {
          ahead_pass = 0;
          if (++ahead_t < n_my) ahead.next(c, a);
        }
      }
    };
    if (MODE != kAnyRot) fetch();
#pragma unroll 1
    for (int t = 0; t < n_my; ++t) {
      const int buf = t & 1;
      uint8_t* const X = sX + buf * 2 * kPart;
      const int base = at.base(), lo = at.lo(), hi = at.hi();
#pragma unroll 1
      for (int pass = 0; pass < 4; ++pass) {
        const int r = (tid >> 3) + 32 * pass;
        const bool live = r >= lo && r < hi;
        float x[16], undo, up;
        float mx = 0.f;                        // of the row before it is rotated: at most sqrt(2) off; NaN is passed over,
                                               // an infinity makes its row NaN
        if (MODE != kAnyRot) {
          if (live) mx = fmaxf(ra.amax(), rb.amax());
#pragma unroll
          for (int o = 4; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
          up = norm_up(mx, undo);
          if (live) {
            ra.scale(up);
            rb.scale(up);
            ra.get(x);
            rb.get(x + 8);
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = 0.f;
          }
          fetch();
          if (live && turned) {
            const float* cs = a.rope.cs + (size_t)(base + r) * rot + 8 * j8;
            float cc[8], ss[8];
            load8(cs, cc);
            load8(cs + half, ss);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int ia = MODE == kPairs ? 2 * e : e, ib = MODE == kPairs ? 2 * e + 1 : 8 + e;
              const float u = x[ia], v = x[ib];
              x[ia] = u * cc[e] - v * ss[e];
              x[ib] = v * cc[e] + u * ss[e];
            }
          }
        } else {
          const T* src = static_cast<const T*>(a.k_new) + (size_t)(at.token + base + r - at.start) * a.ks.row +
                         (size_t)h * a.ks.head;
          const float* cs = a.rope.cs + (size_t)(base + r) * rot;
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int i = 16 * j8 + e;
            float v = live ? Elem<T>::load(src + i) * kDown : 0.f;
            if (live && i < rot) {
              const bool first = a.rope.interleaved ? (i & 1) == 0 : i < half;
              const int j = a.rope.interleaved ? i >> 1 : (first ? i : i - half);
              const int o = a.rope.interleaved ? i ^ 1 : (first ? i + half : i - half);
              const float cc = __ldg(cs + j), ss = __ldg(cs + half + j), z = Elem<T>::load(src + o) * kDown;
              v = first ? v * cc - z * ss : v * cc + z * ss;
            }
            x[e] = v;
            mx = fmaxf(mx, fabsf(v));
          }
#pragma unroll
          for (int o = 4; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
          up = norm_up(mx, undo);
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] *= up;
        }
        if (pass == 0 && t >= 2) tile_wait(&ms.x_free[buf], ((t - 2) >> 1) & 1, ms, c.ctrl);
        if (j8 == 0) ms.unit[t & 3][r] = undo * p_undo * (MODE == kAnyRot ? 1.f / kDown : 1.f);
        uint32_t hw[8], lw[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          hw[e] = split_pair(x[2 * e], x[2 * e + 1]);
          lw[e] = pack_half2(x[2 * e], x[2 * e + 1]);
        }
        *reinterpret_cast<uint4*>(X + part_off(r, da)) = make_uint4(hw[0], hw[1], hw[2], hw[3]);
        *reinterpret_cast<uint4*>(X + part_off(r, db)) = make_uint4(hw[4], hw[5], hw[6], hw[7]);
        *reinterpret_cast<uint4*>(X + kPart + part_off(r, da)) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
        *reinterpret_cast<uint4*>(X + kPart + part_off(r, db)) = make_uint4(lw[4], lw[5], lw[6], lw[7]);
      }
      fence_proxy_async_smem();
      mbar_arrive(&ms.x_full[buf]);
      if (t + 1 < n_my) at.next(c, a);
    }
  } else if (w == kProdWarp) {
    // ================= products =================
    if (lane == 0) {
      const uint32_t idesc = (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | ((uint32_t)(kTile >> 4) << 24);
#pragma unroll 1
      for (int t = 0; t < n_my; ++t) {
        const int buf = t & 1;
        bool ok = mbar_wait_bounded(&ms.x_full[buf], (t >> 1) & 1);
        if (ok && t >= 2) ok = mbar_wait_bounded(&ms.d_free[buf], ((t - 2) >> 1) & 1);
        if (!ok) {
          if (!*(volatile int*)&ms.abort) record_status(c.ctrl, AQUA_ERR_TIMEOUT);
          *(volatile int*)&ms.abort = 1;
          break;
        }
        fence_proxy_async_smem();
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t xa = smem_u32(sX) + buf * 2 * kPart, pa = smem_u32(sP);
#pragma unroll
        for (int pr = 0; pr < 4; ++pr) {     // x_l P_l, x_l P_h, x_h P_l, x_h P_h: the small ones first
          const uint64_t ad = desc_sw128(xa + (pr < 2 ? kPart : 0), 16);
          const uint64_t bd = desc_sw128(pa + (pr % 2 == 0 ? kPart : 0), kTile * 128);
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            mma_f16(tmem + buf * 2 * D + (ks >> 2) * D, ad + (uint64_t)(((ks >> 2) * (kTile * 128) + (ks & 3) * 32) >> 4),
                    bd + (uint64_t)((ks * 16 * 128) >> 4), idesc, pr > 0 || (ks & 3));
        }
        commit_to(&ms.x_free[buf]);
        commit_to(&ms.d_full[buf]);
      }
    }
    __syncwarp();
  } else if (w < kValWarp0) {
    // ================= projected keys: scales, codes, pages =================
    const int kt = tid - kKeyWarp0 * 32, kr = 32 * (w & 3) + lane, kg = kr >> 4;           // slot, its group of 16
    const int per = 1 << (c.page_log2 - 4), g0 = kg & ~(per - 1), mask = (1 << c.page_log2) - 1;
    const uint32_t bytes = (uint32_t)c.m << c.page_log2, block = (uint32_t)((c.m + 31) & ~31) << c.page_log2;   // of a page's keys
#pragma unroll 1
    for (int t = 0; t < n_my; ++t) {
      const int buf = t & 1, lo = at.lo(), hi = at.hi();
      // this slot's page; the page the run starts inside (uniform), with its old scale, read before anyone changes it
      const int pid = at.page_of(c, kg);
      const int open_fill = at.held(c, lo >> 4), open = open_fill > 0 ? at.page_of(c, lo >> 4) : -1;
      const float open_scale = open >= 0 ? c.ks[(size_t)open * c.Hkv + h] : 0.f;
      tile_wait(&ms.d_full[buf], (t >> 1) & 1, ms, c.ctrl);
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      // tensor memory is read twice, for the maxima and for the codes: 128 numbers do not fit the registers
      const uint32_t col = tmem + ((uint32_t)(32 * (w & 3)) << 16) + buf * 2 * D;
      const float unit = ms.unit[t & 3][kr];
      float km = 0.f;
#pragma unroll 1
      for (int q = 0; q < D; q += 32) {
        uint32_t x[32], y[32];
        tmem_ld32(col + q, x);
        tmem_ld32(col + D + q, y);
        tmem_wait_ld(x, y);
        float m = 0.f;
#pragma unroll
        for (int e = 0; e < 32; ++e) m = fmaxf(m, fabsf(__uint_as_float(x[e]) + __uint_as_float(y[e])));
        if (__any_sync(0xffffffffu, !(m * unit < INFINITY))) {   // an infinity in one of the warp's rows: the largest finite ones
          m = 0.f;                           // (by the whole warp: the loads from tensor memory are its joint business)
#pragma unroll 1
          for (int e = 0; e < 32; ++e) {
            uint32_t z0, z1;
            asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(z0) : "r"(col + q + e) : "memory");
            asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(z1) : "r"(col + D + q + e) : "memory");
            asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
            asm volatile("" : "+r"(z0), "+r"(z1));
            const float k = fabsf(__uint_as_float(z0) + __uint_as_float(z1));
            if (k * unit < INFINITY) m = fmaxf(m, k);
          }
        }
        km = fmaxf(km, m);
      }
      km *= unit;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) km = fmaxf(km, __shfl_xor_sync(0xffffffffu, km, o));
      if ((lane & 15) == 0) ms.kgroup[buf][kg] = km;
      named_bar_sync(kBarKey, kKeyThreads);  // the other buffer's readers are past the next barrier by the time it is reused
#pragma unroll 1
      for (int g = g0; g < g0 + per; ++g) km = fmaxf(km, ms.kgroup[buf][g]);
      const float s = page_scale(km, open_scale, pid == open ? open_fill : 0), f = unit / s;
      uint8_t* const codes = sC + buf * (D * kTile);
      {
        uint8_t* dst = codes + (uint32_t)(kr >> c.page_log2) * block + (kr & mask);
        const int row = 1 << c.page_log2;    // bytes from a dimension to the next
#pragma unroll 1
        for (int q = 0; q < c.m; q += 32) {
          uint32_t x[32], y[32];
          tmem_ld32(col + q, x);
          tmem_ld32(col + D + q, y);
          tmem_wait_ld(x, y);
          uint8_t* d = dst + q * row;
#pragma unroll
          for (int e = 0; e < 32; e += 2) {  // dims past d_store fall into the buffer's padding
            const uint16_t code = f32x2_to_e4m3x2((__uint_as_float(x[e]) + __uint_as_float(y[e])) * f,
                                                  (__uint_as_float(x[e + 1]) + __uint_as_float(y[e + 1])) * f);
            d[e * row] = (uint8_t)code;
            d[(e + 1) * row] = (uint8_t)(code >> 8);
          }
        }
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        mbar_arrive(&ms.d_free[buf]);
      }
      // one thread of each page writes its scale: that of the page's first slot in the tile, or the run's first
      const int first = max(lo, 16 * g0);
      if (kr == first && kr < hi && pid >= 0) c.ks[(size_t)pid * c.Hkv + h] = s;
      if (open >= 0) {                       // what the open page holds follows its scale
        const int o0 = (lo >> 4) & ~(per - 1);
        float om = 0.f;
#pragma unroll 1
        for (int g = o0; g < o0 + per; ++g) om = fmaxf(om, ms.kgroup[buf][g]);
        const float now = page_scale(om, open_scale, open_fill);
        if (now != open_scale)
          recode_keys(c.k + c.kblock(open, h), c.m, c.page_log2, open_fill, open_scale / now, kt, kKeyThreads);
      }
      fence_proxy_async_smem();
      named_bar_sync(kBarKey, kKeyThreads);
      // out: whole pages by one bulk copy each, as they lie; pages with other slots in bytes
#pragma unroll 1
      for (int pg = 0; pg < kTile >> c.page_log2; ++pg) {
        const int s0 = pg << c.page_log2, s1 = s0 + mask + 1;
        if (s1 <= lo || s0 >= hi) continue;
        const int pd = at.page_of(c, s0 < lo ? lo >> 4 : s0 >> 4);
        if (pd < 0) continue;
        uint8_t* dst = c.k + c.kblock(pd, h);
        const uint8_t* src = codes + (uint32_t)pg * block;
        if (s0 >= lo && s1 <= hi) {
          if (kt == 0)
            asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes)
                         : "memory");
        } else {
          const int a0 = max(lo, s0) - s0, a1 = min(hi, s1) - s0, lg = c.page_log2 - 4;
#pragma unroll 1
          for (int i = kt; i < c.m << lg; i += kKeyThreads) {                // sixteen slots of a dimension
            const int x0 = (i & ((1 << lg) - 1)) << 4, x1 = x0 + 16;
            if (x0 >= a0 && x1 <= a1) {
              reinterpret_cast<uint4*>(dst)[i] = reinterpret_cast<const uint4*>(src)[i];
            } else if (x0 < a1 && x1 > a0) {
#pragma unroll 1
              for (int x = max(x0, a0); x < min(x1, a1); ++x) dst[16 * i - x0 + x] = src[16 * i - x0 + x];
            }
          }
        }
      }
      if (kt == 0) {
        // the copies of the tile before have read their buffer, which the next tile's codes go to
        asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group.read 1;" ::: "memory");
      }
      if (t + 1 < n_my) at.next(c, a);
    }
    if (kt == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  } else {
    // ================= values =================
    const int vt = tid - kValWarp0 * 32, vw = vt >> 5, col = 8 * (vt & 15);      // sixteen lanes a row: rows 16 i + vt / 16
#pragma unroll 1
    for (int t = 0; t < n_my; ++t) {
      const int base = at.base(), lo = at.lo(), hi = at.hi();
      // the first warp, four lanes to a group of 16 slots: its page, what that held, its old scale
      int pid = -1, fill = 0;
      float old = 0.f;
      const int vg = vt >> 2;
      if (vw == 0) {
        pid = at.page_of(c, vg);
        fill = at.held(c, vg);
        if (pid >= 0 && fill > 0) old = c.vs[(size_t)pid * c.Hkv + h];
      }
      const T* src = static_cast<const T*>(a.v_new) + (size_t)h * a.vs.head + col;
      const long long row0 = (long long)at.token + base - at.start;              // input row of slot 0 (may lie before the run)
      const T* mine = src + (row0 + (vt >> 4)) * a.vs.row;                        // this thread's row of group 0
      // row i of this thread belongs to group i; bf16 rows stay in registers, of f32 rows every second four are
      // loaded again for the codes
      constexpr int kHold = sizeof(T) == 2 ? kGroups : kGroups / 2;
      Raw8<T> rows[kHold];
      auto in_run = [&](int i) { return 16 * i + (vt >> 4) >= lo && 16 * i + (vt >> 4) < hi; };
      auto load_rows = [&](int q) {
#pragma unroll
        for (int i = 0; i < kHold; ++i)
          if (in_run(q + i)) rows[i].load(mine + (size_t)(16 * (q + i)) * a.vs.row);
      };
#pragma unroll
      for (int q = 0; q < kGroups; q += kHold) {
        load_rows(q);
#pragma unroll
        for (int i = 0; i < kHold; ++i) {
          float m = in_run(q + i) ? rows[i].amax() : 0.f;
          if (!(m < INFINITY)) m = finite_amax8(mine + (size_t)(16 * (q + i)) * a.vs.row);
          const uint32_t u = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
          if (lane == 0) ms.vgroup[vw][q + i] = __uint_as_float(u);
        }
      }
      named_bar_sync(kBarVal, kValThreads);
      if (vw == 0) {
        static_assert(kGroups * 4 == 32 && kValThreads == 256, "four lanes a group, two warps' maxima each");
        float m = fmaxf(ms.vgroup[2 * (lane & 3)][vg], ms.vgroup[2 * (lane & 3) + 1][vg]);
        const int per = 1 << (c.page_log2 - 4);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1)     // over the warps' maxima, then over the groups of a page
          if (o < 4 * per) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float s = page_scale(m, old, fill);
        if ((lane & 3) == 0) {
          ms.vinv[vg] = 1.f / s;
          ms.vpid[vg] = pid;
          // one group of each page speaks for it: the page's first, or the run's
          const bool speaks = pid >= 0 && vg == max(vg & ~(per - 1), lo >> 4);
          if (speaks) c.vs[(size_t)pid * c.Hkv + h] = s;
          if (vg == lo >> 4) ms.vrecode = pid >= 0 && fill > 0 ? old / s : 1.f;
        }
      }
      named_bar_sync(kBarVal, kValThreads);
      {
        const int og = lo >> 4, open = ms.vpid[og];
        if (ms.vrecode != 1.f && open >= 0)
          recode_values(c.v + c.vblock(open, h), at.start & ((1 << c.page_log2) - 1), ms.vrecode, vt, kValThreads);
      }
      const int mask = (1 << c.page_log2) - 1;
#pragma unroll
      for (int y = 0; y < kGroups; y += kHold) {
        const int q = kGroups - kHold - y;    // the rows loaded last first
        if (y > 0) load_rows(q);
#pragma unroll
        for (int i = 0; i < kHold; ++i) {
          const int pd = ms.vpid[q + i];
          if (!in_run(q + i) || pd < 0) continue;
          const float s = ms.vinv[q + i];
          float f[8];
          rows[i].get(f);
          *reinterpret_cast<uint2*>(c.v + c.vblock(pd, h) + (size_t)((base + 16 * (q + i) + (vt >> 4)) & mask) * D + col) =
              make_uint2(f32x4_to_e4m3x4(f[0] * s, f[1] * s, f[2] * s, f[3] * s),
                         f32x4_to_e4m3x4(f[4] * s, f[5] * s, f[6] * s, f[7] * s));
        }
      }
      named_bar_sync(kBarVal, kValThreads);
      if (t + 1 < n_my) at.next(c, a);
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (w == kProdWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
}

template <typename T, int MODE>
int launch_tiles_as(const PagedView& c, const AppendParams& a, cudaStream_t st) {
  const int smem = 6 * kPart + 2 * D * kTile + (int)sizeof(TileMisc);
  const int rc = set_smem_limit(paged_append_tile_kernel<T, MODE>, smem, "paged_append_tile_kernel");
  if (rc != AQUA_OK) return rc;
  // a run of n >= 1 tokens touches at most (n - 2) / 128 + 2 tiles, and at most n
  const long long by_tile = a.n_tokens / kTile + 2LL * c.B, most = by_tile < a.n_tokens ? by_tile : a.n_tokens;
  const int each = device_sm_count() / c.Hkv > 0 ? device_sm_count() / c.Hkv : 1;      // blocks a head
  const cudaError_t e = launch_pdl(paged_append_tile_kernel<T, MODE>, dim3((unsigned)(most < each ? most : each), c.Hkv),
                                   dim3(kTileThreads), smem, st, c, a);
  if (e != cudaSuccess) return set_error(AQUA_ERR_CUDA, "paged_append_tile_kernel: %s", cudaGetErrorString(e));
  return check_launch("paged_append_tile_kernel");
}
template <typename T>
int launch_tiles(const PagedView& c, const AppendParams& a, cudaStream_t st) {
  if (a.rope.cs == nullptr) return launch_tiles_as<T, kHalves>(c, a, st);
  if (a.rope.rot % 16 != 0) return launch_tiles_as<T, kAnyRot>(c, a, st);
  return a.rope.interleaved ? launch_tiles_as<T, kPairs>(c, a, st) : launch_tiles_as<T, kHalves>(c, a, st);
}

// One new token for each sequence: a block takes up to kStepGroup sequences of one
// KV head.  Bound by latency: P (64 KB, from L2) is read once per block into
// registers and kept there as f64, whose
// 64 multiply-adds a cycle and SM are enough here; the sums are then exact to f32
// rounding, so that a code differs from the exact one only on a tie.  Warp t
// writes token t.  One sequence 4.8 us, 256 of 8 heads 11.0 us, launches replayed
// from a graph.
constexpr int kStepThreads = 512;
constexpr int kStepGroup = 16;
constexpr int kStepSlices = kStepThreads / D;              // slices of 32 input dims

template <typename T>
__global__ void __launch_bounds__(kStepThreads) paged_append_step_kernel(PagedView c, AppendParams a, int group) {
  extern __shared__ __align__(16) double part[];           // [kStepSlices][group][D]
  __shared__ __align__(16) double xs[kStepGroup][D];       // rotated rows
  __shared__ __align__(16) float raw[kStepGroup][D];
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, h = blockIdx.y;
  const int col = tid & (D - 1), sl = tid >> 7;
  constexpr int R = D / kStepSlices;
  prefetch_head(a.P + (size_t)h * D * D, tid, kStepThreads);
  pdl_wait();
  float pf[R];
  {
    const float* Pg = a.P + ((size_t)h * D + sl * R) * D + col;
#pragma unroll
    for (int i = 0; i < R; ++i) pf[i] = __ldg(Pg + (size_t)i * D);
  }
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
  // enough sequences a block that the blocks fit the SMs at once (152 blocks of 256 sequences, 8 heads: 13.4 us;
  // 144: 10.2)
  const int each = device_sm_count() / c.Hkv > 0 ? device_sm_count() / c.Hkv : 1;     // blocks a head
  const int want = (c.B + each - 1) / each, group = want < kStepGroup ? want : kStepGroup;
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
  // a run of n >= 1 tokens touches at most (n - 2) / page + 2 pages, and at most n (of runs that share no rows)
  const long long by_page = a.n_tokens / (1 << c.page_log2) + 2LL * c.B;
  const int segs = (int)(by_page < a.n_tokens ? by_page : a.n_tokens);
  // no more blocks than run at once, two an SM: each reads P once (304 segments of 16 heads: 49 us with a block each)
  const int each = 2 * device_sm_count() / c.Hkv > 0 ? 2 * device_sm_count() / c.Hkv : 1;
  paged_append_run_kernel<T><<<dim3(segs < each ? segs : each, c.Hkv), kThreads, smem, st>>>(c, a);
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
  // Estimates in ns, from both kernels measured over 1 to 128 runs of 16 to 512 tokens, pages of 16 to 128 and 1 and
  // 8 heads.  CUDA cores: 0.3 us a token, of a page's worth of one block or of an SM's share; tiles: a fixed 10 us
  // and 5.5 us for every further tile of an SM, however few of its rows are used.  (64 tokens of one sequence, 8
  // heads, pages of 64: 21.5 us against 17; 16 tokens: 7.5 against 13.)
  const long long sms = device_sm_count(), run = n_tokens / c.B + 1, page = 1 << c.page_log2;
  const long long share = n_tokens * (long long)c.Hkv / sms, most = run < page ? run : page;
  const long long cores = 4000 + 300 * (share > most ? share : most);
  const long long tiles = 10000 + 5500 * ((n_tokens / kTile + c.B) * (long long)c.Hkv / sms);
  if (tiles < cores) return bf16 ? launch_tiles<__nv_bfloat16>(c, a, st) : launch_tiles<float>(c, a, st);
  return bf16 ? launch_run<__nv_bfloat16>(c, a, st) : launch_run<float>(c, a, st);
}

}  // namespace aqua
