// One decode step of AQUA attention over the paged 8-bit cache.
//
// paged_select_kernel, one block per (sequence b, KV head g): for the group's
// query heads q~ = rope(q, len - 1) P (f64, rounded once), the k largest |q~_j|
// (ties to the lower j), the union U of the kept dimensions, and the masked
// queries in the layout the tensor cores take them.
//
// paged_attend_kernel, persistent: the tokens of all (b, g) are cut into tiles
// of 128 and the flat sequence of tiles is split evenly over the blocks.  Per
// tile the |U| kept key rows (16 tokens a chunk, from whatever page holds them)
// and the value rows are gathered into shared memory, several tiles ahead; each
// of the four warps owns 32 tokens and keeps a running softmax of its own:
//
//   s_t  = ks(page) sum_{j in U} q~_j code_t[j] / sqrt(d)        S^T = K^T q on mma m16n8k16
//   w_t  = s_t log2(e) + log2 vs(page),   p_t = 2^(w_t - M),  M the running max of w
//   O   += p_t code_t[v],                 l += p_t / vs(page)    O^T = V^T p^T on mma m16n8k16
//   out  = O / l,   lse = ln2 (M + log2 l)
//
// Taking the value scale into the exponent makes O a plain sum over codes, so
// pages with different scales share one accumulator, and what weighs most in O
// has p = 1.  e4m3 codes are exact in f16; q~ and p enter as two f16 parts
// (columns 2h and 2h + 1 of the eight-column operand), 22 bits together.
// A block that starts or ends inside a (b, g) writes (M, l, O);
// paged_merge_kernel adds the parts in block order, so results do not depend on timing.
//
// edgentiq, "How AQUA Works", Online Inference: scores on the selected
// dimensions, softmax, weighted sum of the unprojected values.
#include <math.h>

#include "paged_internal.cuh"

namespace aqua {

namespace {

constexpr int D = kHeadDim;
constexpr int TT = 128;                    // tokens per tile
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 3;
constexpr int kCtasPerSm = 2;
constexpr int kMaxG = 8;
constexpr int kSelThreads = 512;

struct DecodeP {
  const int32_t* len;
  const void* q;
  Strides qs;
  const float* P;
  RopeView rope;
  int Hq, k;
  float scale;
  void* out;
  int out_bf16;
  int32_t* sel_out;
  float* qproj_out;
  float* lse_out;
  // workspace
  int32_t* ucount;       // [n_units] kept rows
  uint8_t* ulist;        // [n_units][D] kept rows, see ulist_slot
  uint2* qfrag;          // [n_units][8][NT][32] masked queries, B operand of the score product
  float* qfac;           // [n_units][kMaxG] factor of a head's scores (log2 domain, without the key scale)
  float2* part_ml;       // [2 * blocks][kMaxG] (M, l) of a partial result
  float* part_o;         // [2 * blocks][kMaxG][D]
  int4* split;           // [blocks] block x starts inside unit .x, whose tiles lie in blocks .y ... .z; .w: slot of
                         // block .y's part; .x < 0: x starts with a unit
};

// Row r of the union is loaded by threads r % 16 (groups of eight threads), as
// that group's row r / 16: the eight rows of a group lie side by side.
__device__ __forceinline__ int ulist_slot(int r) { return (r & 15) * 8 + (r >> 4); }

__device__ __forceinline__ int n_tiles(int len) { return (len + TT - 1) / TT; }

__device__ __forceinline__ int seq_tokens(const PagedView& c, const DecodeP& p, int b) {
  bool bad;
  return checked_len(__ldg(p.len + b), c, p.rope.cs ? p.rope.n_pos : 0x7fffffff, bad);
}

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ void store_out_elem(const DecodeP& p, size_t i, float v) {
  if (p.out_bf16)
    static_cast<__nv_bfloat16*>(p.out)[i] = __float2bfloat16_rn(v);
  else
    static_cast<float*>(p.out)[i] = v;
}

// result of a softmax sum: no visible token gives 0 and -inf, NaN stays
__device__ __forceinline__ float normalised(float O, float L) { return L == 0.f ? 0.f : O / L; }
__device__ __forceinline__ float lse_of(float M, float L) { return L == 0.f ? -INFINITY : kLn2 * (M + log2f(L)); }

// ============================================================================
// rotation, projection, top-k
// ============================================================================

// GP: the group size padded to 1, 2, 4 or 8 (rows G .. GP-1 are zeros and never stored).
template <typename T, int GP>
__global__ void __launch_bounds__(kSelThreads) paged_select_kernel(PagedView c, DecodeP p, int G, int NT) {
  constexpr int kSlices = kSelThreads / D, kRows = D / kSlices;      // P rows per thread
  __shared__ __align__(16) double qd[GP][D];       // rotated rows; later the ranking keys
  __shared__ double part[kSlices][GP][D];
  __shared__ float qs[GP][D];                      // raw rows; later the kept q~, 0 elsewhere
  float (*raw)[D] = qs;
  uint32_t (*key)[D] = reinterpret_cast<uint32_t (*)[D]>(&qd[0][0]);
  __shared__ uint32_t kept[GP][4];
  __shared__ float qmul[GP];
  __shared__ int urow[D];
  const int u = blockIdx.x, b = u / c.Hkv, g = u % c.Hkv;
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  const int j = tid & 127, sl = tid >> 7;
  // P is read before the wait on the previous kernel: whatever may still run then does not write it
  float pr[kRows];
  {
    const float* Pg = p.P + (size_t)g * D * D + (size_t)sl * kRows * D + j;
#pragma unroll
    for (int i = 0; i < kRows; ++i) pr[i] = __ldg(Pg + i * D);
  }
  pdl_wait();
  pdl_launch_dependents();
  const int len = __ldg(p.len + b);
  bool bad;
  const int n = checked_len(len, c, p.rope.cs ? p.rope.n_pos : 0x7fffffff, bad);
  if (tid == 0 && bad) report_arg(c);
  const T* q = static_cast<const T*>(p.q) + (size_t)b * p.qs.row + (size_t)g * G * p.qs.head;
  for (int i = tid; i < GP * D; i += kSelThreads)
    raw[i >> 7][i & 127] = (i >> 7) < G ? Elem<T>::load(q + (size_t)(i >> 7) * p.qs.head + (i & 127)) : 0.f;
  __syncthreads();
  for (int i = tid; i < GP * D; i += kSelThreads) {
    const int hh = i >> 7;
    double x = raw[hh][j];
    if (p.rope.cs != nullptr && n > 0) {
      const float* cs = p.rope.cs + (size_t)(n - 1) * p.rope.rot;
      const int rot = p.rope.rot, half = rot >> 1;
      if (j < rot) {
        const bool first = p.rope.interleaved ? (j & 1) == 0 : j < half;
        const int a = p.rope.interleaved ? j >> 1 : (first ? j : j - half);
        const int o = p.rope.interleaved ? j ^ 1 : (first ? j + half : j - half);
        const double cc = __ldg(cs + a), ss = __ldg(cs + half + a), y = raw[hh][o];
        x = first ? x * cc - y * ss : x * cc + y * ss;
      }
    }
    qd[hh][j] = x;
  }
  __syncthreads();
  {
    // partial sums over kRows input dims of column j, all heads of the group
    double acc[GP];
#pragma unroll
    for (int hh = 0; hh < GP; ++hh) acc[hh] = 0.0;
#pragma unroll
    for (int i = 0; i < kRows; i += 2) {
      const double x0 = pr[i], x1 = pr[i + 1];
#pragma unroll
      for (int hh = 0; hh < GP; ++hh) {
        const double2 qv = *reinterpret_cast<const double2*>(&qd[hh][sl * kRows + i]);
        acc[hh] = fma(x1, qv.y, fma(x0, qv.x, acc[hh]));
      }
    }
#pragma unroll
    for (int hh = 0; hh < GP; ++hh) part[sl][hh][j] = acc[hh];
  }
  __syncthreads();
  for (int i = tid; i < GP * D; i += kSelThreads) {
    const int hh = i >> 7;
    double sum = part[0][hh][j];
#pragma unroll
    for (int x = 1; x < kSlices; ++x) sum += part[x][hh][j];
    const float qt = (float)sum;
    qs[hh][j] = qt;
    // magnitude order as unsigned order; dims past d_store below every candidate, NaN payloads one key
    key[hh][j] = j < c.m ? min(__float_as_uint(fabsf(qt)), 0x7F800001u) + 1u : 0u;
    if (p.qproj_out && hh < G) p.qproj_out[((size_t)b * p.Hq + (size_t)g * G) * D + i] = qt;
  }
  __syncthreads();
  // Dimension j is kept when fewer than k others rank before it (larger, or equal and lower).  Four
  // warps a head count the larger ones; equal keys are looked at only if they straddle the cut.
  for (int hh = sl; hh < G; hh += kSlices) {
    const uint32_t kj = key[hh][j];
    int rank = 0;
#pragma unroll 8
    for (int x = 0; x < D; x += 4) {
      const uint4 o = *reinterpret_cast<const uint4*>(&key[hh][x]);
      rank += (int)(o.x > kj) + (int)(o.y > kj) + (int)(o.z > kj) + (int)(o.w > kj);
    }
    const int in = named_bar_popc(2 + sl, D, j < c.m && rank < p.k);
    if (in > p.k) {
      for (int x = 0; x < j; ++x) rank += key[hh][x] == kj;
    }
    const uint32_t bal = __ballot_sync(0xffffffffu, j < c.m && rank < p.k);
    if (lane == 0) kept[hh][w & 3] = bal;
  }
  __syncthreads();
  // masked rows, their selected dims, and each head's power-of-two normaliser
  for (int i = tid; i < G * D; i += kSelThreads) {
    const int hh = i >> 7, wd = j >> 5;
    const uint32_t word = kept[hh][wd];
    if ((word >> (j & 31)) & 1u) {
      if (p.sel_out) {
        int pos = __popc(word & ((1u << (j & 31)) - 1u));
        for (int x = 0; x < wd; ++x) pos += __popc(kept[hh][x]);
        p.sel_out[((size_t)b * p.Hq + (size_t)g * G + hh) * p.k + pos] = j;
      }
    } else {
      qs[hh][j] = 0.f;
    }
  }
  if (tid < D) {
    uint32_t um[4];
#pragma unroll
    for (int wd = 0; wd < 4; ++wd) {
      um[wd] = 0;
      for (int hh = 0; hh < G; ++hh) um[wd] |= kept[hh][wd];
    }
    const int count = __popc(um[0]) + __popc(um[1]) + __popc(um[2]) + __popc(um[3]);
    urow[tid] = -1;
    named_bar_sync(1, D);
    if ((um[tid >> 5] >> (tid & 31)) & 1u) {
      int r = __popc(um[tid >> 5] & ((1u << (tid & 31)) - 1u));
      for (int x = 0; x < (tid >> 5); ++x) r += __popc(um[x]);
      urow[r] = tid;
    }
    named_bar_sync(1, D);
    p.ulist[(size_t)u * D + ulist_slot(tid)] = (uint8_t)(urow[tid] < 0 ? 0 : urow[tid]);
    if (tid == 0) p.ucount[u] = count;
  }
  __syncthreads();
  if (w < G) {
    float mx = 0.f;
#pragma unroll
    for (int x = 0; x < 4; ++x) mx = fmaxf(mx, finite_abs(qs[w][lane + 32 * x]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    // 2^-e with mx = f 2^e: the largest part lies in [1, 2), far from f16's ends
    const int e = min(max((int)(__float_as_uint(mx) >> 23) - 127, -100), 100);
    if (lane == 0) {
      qmul[w] = __uint_as_float((uint32_t)(127 - e) << 23);
      p.qfac[(size_t)u * kMaxG + w] = __uint_as_float((uint32_t)(127 + e) << 23) * p.scale * kLog2e;
    }
  }
  __syncthreads();
  // B operand of the score product: column 2h holds the high and 2h + 1 the low f16 part of head h;
  // k index 2t + e of a step of 16 rows is row 4t + e, index 2t + 8 + e row 4t + 2 + e
  for (int i = tid; i < 8 * NT * 32; i += kSelThreads) {
    const int ln = i & 31, nt = (i >> 5) % NT, ks = (i >> 5) / NT;
    const int col = ln >> 2, t = ln & 3, hh = 4 * nt + (col >> 1);
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (hh < G) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int d = urow[16 * ks + 4 * t + e];
        if (d >= 0) {
          const float x = qs[hh][d] * qmul[hh];
          const float hi = __half2float(__float2half_rn(x));
          v[e] = (col & 1) ? x - hi : hi;
        }
      }
    }
    p.qfrag[(((size_t)u * 8 + ks) * NT + nt) * 32 + ln] = make_uint2(pack_f16(v[0], v[1]), pack_f16(v[2], v[3]));
  }
  // an empty sequence has no tiles: attention over no token is 0 with lse -inf
  if (n == 0) {
    const size_t r0 = (size_t)b * p.Hq + (size_t)g * G;
    for (int i = tid; i < G * D; i += kSelThreads) store_out_elem(p, r0 * D + i, 0.f);
    if (p.lse_out && tid < G) p.lse_out[r0 + tid] = -INFINITY;
  }
}

// ============================================================================
// attention
// ============================================================================

// Shared memory of one stage: the tile's key rows, its value rows, its scales.
constexpr int kStageV = D * TT;                       // bytes of V ahead of the key rows
struct TileMeta {
  int pid[TT / 16];        // page of every 16 tokens, -1: none
  float ks[TT / 16];       // its key scale; negative: no page
  float vs[TT / 16];
};
// A tile's page ids are staged one step before its copies are issued, kStages - 1
// tiles ahead of the one being consumed: kStages + 1 sets are live at once.
constexpr int kMeta = kStages + 1;

// Position in the flat sequence of tiles.
struct Cursor {
  int u;                   // unit (b * Hkv + g)
  int b, g;
  int len;                 // tokens of the sequence
  int tile;                // tile of the unit
};

__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? 16 : 0;
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Next unit with tokens after cur (its tiles are used up).
__device__ __forceinline__ void next_unit(const PagedView& c, const DecodeP& p, Cursor& cur) {
  cur.tile = 0;
  ++cur.u;
  if (++cur.g < c.Hkv) return;
  cur.g = 0;
  do {
    ++cur.b;
    cur.len = cur.b < c.B ? seq_tokens(c, p, cur.b) : 0;
  } while (cur.b < c.B && cur.len == 0);
  cur.u = cur.b * c.Hkv;
}

template <int NT>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) paged_attend_kernel(PagedView c, DecodeP p, int G) {
  extern __shared__ __align__(128) uint8_t dyn[];
  const int stage_bytes = kStageV + ((c.m + 15) & ~15) * TT;
  __shared__ TileMeta meta[kMeta];
  __shared__ float merge_ml[kWarps][kMaxG][2];
  __shared__ long long scan[kWarps + 1];
  __shared__ Cursor s_cur;
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, gr = lane >> 2, tg = lane & 3;

  // ---- this block's share [t0, t1) of the flat tile sequence (the lengths were written before the
  // selection kernel started, which released this one after its own wait)
  long long total = 0;
  for (int base = 0; base < c.B; base += kThreads) {
    const int b = base + tid;
    int x = b < c.B ? n_tiles(seq_tokens(c, p, b)) : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    __syncthreads();
    if (lane == 0) scan[w] = x;
    __syncthreads();
    for (int y = 0; y < kWarps; ++y) total += scan[y];
  }
  total *= c.Hkv;
  const long long nb = min((long long)gridDim.x, total);      // every share has a tile
  if (blockIdx.x >= nb) {
    if (tid == 0) p.split[blockIdx.x].x = -1;
    return;
  }
  const long long t0 = blockIdx.x * total / nb, t1 = (blockIdx.x + 1) * total / nb;
  // the unit that holds tile t0
  {
    long long before = 0;
    for (int base = 0; base < c.B; base += kThreads) {
      const int b = base + tid;
      const int len = b < c.B ? seq_tokens(c, p, b) : 0;
      const int x = n_tiles(len);
      int sum = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += y;
      }
      __syncthreads();
      if (lane == 31) scan[w] = sum;
      __syncthreads();
      long long off = before, all = 0;
      for (int y = 0; y < kWarps; ++y) {
        if (y < w) off += scan[y];
        all += scan[y];
      }
      const long long first = (off + sum - x) * c.Hkv, last = (off + sum) * c.Hkv;
      if (x > 0 && t0 >= first && t0 < last) {
        const int r = (int)(t0 - first);
        s_cur.b = b;
        s_cur.g = r / x;
        s_cur.tile = r % x;
        s_cur.u = b * c.Hkv + r / x;
        s_cur.len = len;
      }
      before += all;
    }
    __syncthreads();
  }
  pdl_wait();                               // the selection's results; the merge of an earlier call has read its parts
  pdl_launch_dependents();
  if (tid == 0) {
    int4 sp = make_int4(-1, 0, 0, 0);
    if (s_cur.tile > 0) {
      // the unit's tiles are [f, f + n) of the flat sequence; tile x lies in block ((x + 1) nb - 1) / total
      const long long f = t0 - s_cur.tile, n = n_tiles(s_cur.len);
      const long long first = ((f + 1) * nb - 1) / total, last = ((f + n) * nb - 1) / total;
      sp = make_int4(s_cur.u, (int)first, (int)last, first * total / nb < f ? 1 : 0);
    }
    p.split[blockIdx.x] = sp;
  }

  const int lc = tid & 7, lr = tid >> 3;    // this thread's chunk and first row of every copied tile
  const uint32_t smem0 = smem_u32(dyn);
  const int pmask = (1 << c.page_log2) - 1;

  Cursor ic = s_cur;                        // next tile to issue
  int iu = -1;                              // unit whose rows are in `rows`
  uint2 rows = make_uint2(0, 0);
  int icount = 0;
  const int n_my = (int)(t1 - t0);
  int issued = 0;

  // page of 16 tokens of the tile at the issue cursor (threads 0..7, one chunk each)
  auto page_of_chunk = [&]() {
    int pid = -1;
    const int t = ic.tile * TT + 16 * tid;
    if (tid < TT / 16 && t < ic.len) {
      pid = __ldg(c.table + (size_t)ic.b * c.max_pages + (t >> c.page_log2));
      if (pid < 0 || pid >= c.n_pages) {
        pid = -1;
        report_arg(c);
      }
    }
    return pid;
  };
  auto issue = [&]() {
    TileMeta& md = meta[issued % kMeta];
    if (ic.u != iu) {
      iu = ic.u;
      rows = *reinterpret_cast<const uint2*>(p.ulist + (size_t)iu * D + lr * 8);
      icount = p.ucount[iu];
    }
    const uint32_t vbase = smem0 + (issued % kStages) * stage_bytes, kbase = vbase + kStageV;
    const int tb = ic.tile * TT;
    // values: rows lr, lr + 16, ..., chunk lc of 16 dims; rows past the length are zeros
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = lr + 16 * i, t = tb + r;
      const int pid = md.pid[i];
      const bool ok = pid >= 0 && t < ic.len;
      const uint8_t* src = ok ? c.v + c.vblock(pid, ic.g) + (size_t)(t & pmask) * D + lc * 16 : c.v;
      cp_async16_zfill(vbase + r * D + ((lc ^ (((r >> 3) & 3) * 2)) << 4), src, ok);
    }
    // kept key rows lr, lr + 16, ..., chunk lc of 16 tokens; rows past the union up to the next
    // multiple of 16 are zeros
    const int pid = md.pid[lc];
    const uint8_t* kb = c.k;
    if (pid >= 0) kb += c.kblock(pid, ic.g) + ((tb + 16 * lc) & pmask);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (16 * i >= icount) break;
      const int r = lr + 16 * i;
      const int d = (i < 4 ? rows.x >> (8 * i) : rows.y >> (8 * (i - 4))) & 0xff;
      const bool ok = pid >= 0 && r < icount;
      cp_async16_zfill(kbase + r * TT + ((lc ^ (((r >> 2) & 3) * 2)) << 4), kb + (ok ? (size_t)d << c.page_log2 : 0),
                       ok);
    }
    // scales of the tile's pages
    if (tid < TT / 16) {
      if (pid >= 0) {                       // lc == tid here
        const size_t si = (size_t)pid * c.Hkv + ic.g;
        cp_async_small<4>(&md.ks[tid], c.ks + si);
        cp_async_small<4>(&md.vs[tid], c.vs + si);
      } else {
        md.ks[tid] = -1.f;
        md.vs[tid] = 1.f;
      }
    }
    ++issued;
    if (issued < n_my && ++ic.tile >= n_tiles(ic.len)) next_unit(c, p, ic);
  };

  if (tid < TT / 16) meta[0].pid[tid] = page_of_chunk();
  __syncthreads();
  for (int s = 0; s < kStages - 1; ++s) {
    if (issued < n_my) issue();
    cp_async_commit();
    if (issued < n_my && tid < TT / 16) meta[issued % kMeta].pid[tid] = page_of_chunk();
    __syncthreads();
  }

  // ---- consume
  Cursor cc = s_cur;
  uint2 qf[8][NT];
  float fac[NT];
  float o[NT][8][4];
  float mx[NT], l[NT];
  int nks = 0;
  bool fresh = true;
  const int seg_first = cc.tile;
  int seg_start = seg_first;

  for (int it = 0; it < n_my; ++it) {
    const int st = it % kStages;
    if (fresh) {
      fresh = false;
      nks = (p.ucount[cc.u] + 15) >> 4;
#pragma unroll
      for (int ks = 0; ks < 8; ++ks)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) qf[ks][nt] = p.qfrag[(((size_t)cc.u * 8 + ks) * NT + nt) * 32 + lane];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        fac[nt] = 4 * nt + tg < G ? p.qfac[(size_t)cc.u * kMaxG + 4 * nt + tg] : 0.f;
        mx[nt] = -INFINITY;
        l[nt] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.f;
      }
      seg_start = cc.tile;
    }
    cp_async_wait<kStages - 2>();
    __syncthreads();
    // refill the stage that was consumed in the previous iteration; the page ids of the tile after that
    // are fetched now and stored once this tile is done
    if (issued < n_my) issue();
    cp_async_commit();
    const int stage_next = issued < n_my ? issued % kMeta : -1;
    int next_pid = -1;
    if (stage_next >= 0) next_pid = page_of_chunk();
    // ---- scores of this warp's 32 tokens: token 4 gr + j of the warp is row gr of product j / 2, low
    // half for even j, high half (row gr + 8) for odd j
    uint8_t* vt = dyn + st * stage_bytes;
    const uint8_t* kt = vt + kStageV;
    const int chunk = 2 * w + (gr >> 2);
    const float ksc = meta[it % kMeta].ks[chunk], vsc = meta[it % kMeta].vs[chunk];
    float s[NT][2][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nt][x][e] = 0.f;
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
      if (ks < nks) {
        const uint8_t* kr = kt + (16 * ks + 4 * tg) * TT + ((chunk ^ (2 * tg)) << 4) + 4 * (gr & 3);
        const uint32_t r0 = *reinterpret_cast<const uint32_t*>(kr);
        const uint32_t r1 = *reinterpret_cast<const uint32_t*>(kr + TT);
        const uint32_t r2 = *reinterpret_cast<const uint32_t*>(kr + 2 * TT);
        const uint32_t r3 = *reinterpret_cast<const uint32_t*>(kr + 3 * TT);
        const uint32_t a01 = __byte_perm(r0, r1, 0x5140), a23 = __byte_perm(r0, r1, 0x7362);
        const uint32_t b01 = __byte_perm(r2, r3, 0x5140), b23 = __byte_perm(r2, r3, 0x7362);
        const uint32_t A0[4] = {e4m3x2_to_f16x2((uint16_t)a01), e4m3x2_to_f16x2((uint16_t)(a01 >> 16)),
                                e4m3x2_to_f16x2((uint16_t)b01), e4m3x2_to_f16x2((uint16_t)(b01 >> 16))};
        const uint32_t A1[4] = {e4m3x2_to_f16x2((uint16_t)a23), e4m3x2_to_f16x2((uint16_t)(a23 >> 16)),
                                e4m3x2_to_f16x2((uint16_t)b23), e4m3x2_to_f16x2((uint16_t)(b23 >> 16))};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_f16_16816(s[nt][0], A0, qf[ks][nt].x, qf[ks][nt].y);
          mma_f16_16816(s[nt][1], A1, qf[ks][nt].x, qf[ks][nt].y);
        }
      }
    }
    // ---- running softmax; head 4 nt + tg, tokens 4 gr + {0, 1, 2, 3} of the warp
    const int tok = cc.tile * TT + 32 * w + 4 * gr;
    const bool page_ok = ksc >= 0.f;
    const float lv = __log2f(vsc), iv = 1.f / vsc;
    uint32_t pb[NT][2][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float f = fac[nt] * ksc;
      float x[4];
      x[0] = (s[nt][0][0] + s[nt][0][1]) * f + lv;
      x[1] = (s[nt][0][2] + s[nt][0][3]) * f + lv;
      x[2] = (s[nt][1][0] + s[nt][1][1]) * f + lv;
      x[3] = (s[nt][1][2] + s[nt][1][3]) * f + lv;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (!page_ok || tok + j >= cc.len) x[j] = -INFINITY;
      float m = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
      const float mn = fmaxf(mx[nt], m);
      const float ref = mn == -INFINITY ? 0.f : mn;
      const float al = fast_exp2(mx[nt] - ref);
      mx[nt] = mn;
      l[nt] *= al;
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][i][e] *= al;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float pj = fast_exp2(x[j] - ref);
        l[nt] = fmaf(pj, iv, l[nt]);
        const float hi = __half2float(__float2half_rn(pj));
        pb[nt][j >> 1][j & 1] = movmatrix_trans(pack_f16(hi, pj - hi));
      }
    }
    // ---- O^T += V^T p^T: product x takes the tokens of score product x
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const uint8_t* vr = vt + (32 * w + 8 * tg + 2 * x) * D + ((gr ^ (2 * tg)) << 4);
      const uint4 v0 = *reinterpret_cast<const uint4*>(vr);                 // token 8 tg + 2 x
      const uint4 v2 = *reinterpret_cast<const uint4*>(vr + D);             // + 1: rows 8.. of the k index
      const uint4 v1 = *reinterpret_cast<const uint4*>(vr + 4 * D);         // + 4: the odd k index
      const uint4 v3 = *reinterpret_cast<const uint4*>(vr + 5 * D);
      const uint32_t* p0 = reinterpret_cast<const uint32_t*>(&v0);
      const uint32_t* p1 = reinterpret_cast<const uint32_t*>(&v1);
      const uint32_t* p2 = reinterpret_cast<const uint32_t*>(&v2);
      const uint32_t* p3 = reinterpret_cast<const uint32_t*>(&v3);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t a01 = __byte_perm(p0[q], p1[q], 0x5140), a23 = __byte_perm(p0[q], p1[q], 0x7362);
        const uint32_t b01 = __byte_perm(p2[q], p3[q], 0x5140), b23 = __byte_perm(p2[q], p3[q], 0x7362);
        const uint32_t A0[4] = {e4m3x2_to_f16x2((uint16_t)a01), e4m3x2_to_f16x2((uint16_t)(a01 >> 16)),
                                e4m3x2_to_f16x2((uint16_t)b01), e4m3x2_to_f16x2((uint16_t)(b01 >> 16))};
        const uint32_t A1[4] = {e4m3x2_to_f16x2((uint16_t)a23), e4m3x2_to_f16x2((uint16_t)(a23 >> 16)),
                                e4m3x2_to_f16x2((uint16_t)b23), e4m3x2_to_f16x2((uint16_t)(b23 >> 16))};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_f16_16816(o[nt][2 * q], A0, pb[nt][x][0], pb[nt][x][1]);
          mma_f16_16816(o[nt][2 * q + 1], A1, pb[nt][x][0], pb[nt][x][1]);
        }
      }
    }
    if (stage_next >= 0 && tid < TT / 16) meta[stage_next].pid[tid] = next_pid;

    // ---- end of the unit, or of this block's share of it
    const bool last_tile = cc.tile + 1 == n_tiles(cc.len);
    if (!last_tile && it + 1 < n_my) {
      ++cc.tile;
      continue;
    }
    // merge the four warps (in this tile's value buffer, which is refilled only after the next
    // iteration's barrier): O column pairs, rows d = 16 gr + 2 i (+ 1)
    static_assert(kWarps * kMaxG * D * 4 <= kStageV, "merge buffer");
    float* merge_o = reinterpret_cast<float*>(vt);          // [kWarps][G][D]
    __syncthreads();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float lt = l[nt];
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) lt += __shfl_xor_sync(0xffffffffu, lt, d);
      const int hh = 4 * nt + tg;
      if (hh < G) {
        if (gr == 0) {
          merge_ml[w][hh][0] = mx[nt];
          merge_ml[w][hh][1] = lt;
        }
        float* mo = merge_o + ((size_t)w * G + hh) * D + 16 * gr;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *reinterpret_cast<float2*>(mo + 2 * i) =
              make_float2(o[nt][i][0] + o[nt][i][1], o[nt][i][2] + o[nt][i][3]);
      }
    }
    __syncthreads();
    const bool whole = seg_start == 0 && last_tile;
    const size_t row0 = (size_t)cc.b * p.Hq + (size_t)cc.g * G;
    const int slot = 2 * blockIdx.x + (it + 1 - (cc.tile + 1 - seg_start) > 0 ? 1 : 0);   // 0: the share's first piece
    for (int hh = 0; hh < G; ++hh) {
      float M = -INFINITY;
#pragma unroll
      for (int x = 0; x < kWarps; ++x) M = fmaxf(M, merge_ml[x][hh][0]);
      const float ref = M == -INFINITY ? 0.f : M;
      float L = 0.f, O = 0.f;
#pragma unroll
      for (int x = 0; x < kWarps; ++x) {
        const float f = fast_exp2(merge_ml[x][hh][0] - ref);
        L = fmaf(merge_ml[x][hh][1], f, L);
        O = fmaf(merge_o[((size_t)x * G + hh) * D + tid], f, O);
      }
      if (whole) {
        store_out_elem(p, (row0 + hh) * D + tid, normalised(O, L));
        if (p.lse_out && tid == 0) p.lse_out[row0 + hh] = lse_of(M, L);
      } else {
        p.part_o[((size_t)slot * kMaxG + hh) * D + tid] = O;
        if (tid == 0) p.part_ml[(size_t)slot * kMaxG + hh] = make_float2(M, L);
      }
    }
    __syncthreads();                        // the merge buffers are free again
    if (it + 1 < n_my) {
      fresh = true;
      next_unit(c, p, cc);
    }
  }
  cp_async_wait<0>();
}

// ============================================================================
// merge of the parts of units that several blocks shared
// ============================================================================

// One block per (boundary between two attention blocks, query head of the group);
// the first boundary inside a unit merges it.  Each of eight warps adds every
// eighth part, a float4 of O per lane, then the eight sums are added in order.
constexpr int kMergeWarps = 8;
constexpr int kMaxParts = 2048;

__global__ void __launch_bounds__(kMergeWarps * 32) paged_merge_kernel(PagedView c, DecodeP p, int G) {
  __shared__ float fac[kMaxParts];
  __shared__ __align__(16) float sum[kMergeWarps][D];
  __shared__ float red[2][kMergeWarps];
  const int x = blockIdx.x + 1, hh = blockIdx.y, tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  pdl_wait();
  const int4 sp = p.split[x];
  if (sp.x < 0 || sp.y != x - 1) return;
  const int n = sp.z - sp.y + 1;
  auto slot = [&](int i) { return (size_t)(2 * (sp.y + i) + (i == 0 ? sp.w : 0)) * kMaxG + hh; };
  float M = -INFINITY;
  for (int i = tid; i < n; i += kMergeWarps * 32) M = fmaxf(M, p.part_ml[slot(i)].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if (lane == 0) red[0][w] = M;
  __syncthreads();
#pragma unroll
  for (int y = 0; y < kMergeWarps; ++y) M = fmaxf(M, red[0][y]);
  const float ref = M == -INFINITY ? 0.f : M;
  float L = 0.f;
  for (int i = tid; i < n; i += kMergeWarps * 32) {
    const float2 ml = p.part_ml[slot(i)];
    const float f = fast_exp2(ml.x - ref);
    fac[i] = f;
    L = fmaf(ml.y, f, L);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
  if (lane == 0) red[1][w] = L;
  __syncthreads();
  L = 0.f;
#pragma unroll
  for (int y = 0; y < kMergeWarps; ++y) L += red[1][y];
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int i = w; i < n; i += kMergeWarps) {
    const float4 v = *reinterpret_cast<const float4*>(p.part_o + slot(i) * D + 4 * lane);
    const float f = fac[i];
    acc.x = fmaf(v.x, f, acc.x); acc.y = fmaf(v.y, f, acc.y);
    acc.z = fmaf(v.z, f, acc.z); acc.w = fmaf(v.w, f, acc.w);
  }
  *reinterpret_cast<float4*>(&sum[w][4 * lane]) = acc;
  __syncthreads();
  if (tid < D) {
    float O = 0.f;
#pragma unroll
    for (int y = 0; y < kMergeWarps; ++y) O += sum[y][tid];
    const size_t row = (size_t)(sp.x / c.Hkv) * p.Hq + (size_t)(sp.x % c.Hkv) * G + hh;
    store_out_elem(p, row * D + tid, normalised(O, L));
    if (p.lse_out && tid == 0) p.lse_out[row] = lse_of(M, L);
  }
}

// ---------------------------------------------------------------- host side
struct Layout {
  size_t ucount, ulist, qfrag, qfac, part_ml, part_o, split, total;
};

Layout layout_of(int n_units, int G, int blocks) {
  const int NT = G > 4 ? 2 : 1;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t r = at;
    at = (at + bytes + 255) & ~(size_t)255;
    return r;
  };
  Layout y;
  y.ucount = take((size_t)n_units * 4);
  y.ulist = take((size_t)n_units * D);
  y.qfrag = take((size_t)n_units * 8 * NT * 32 * sizeof(uint2));
  y.qfac = take((size_t)n_units * kMaxG * 4);
  y.part_ml = take((size_t)2 * blocks * kMaxG * sizeof(float2));
  y.part_o = take((size_t)2 * blocks * kMaxG * D * 4);
  y.split = take((size_t)blocks * sizeof(int4));
  y.total = at;
  return y;
}

int attend_blocks() {
  const int n = kCtasPerSm * device_sm_count();
  return n < kMaxParts ? n : kMaxParts;
}

template <typename T>
cudaError_t launch_select(const PagedView& c, const DecodeP& p, int G, int NT, cudaStream_t st) {
  const dim3 grid(c.B * c.Hkv), block(kSelThreads);
  if (G == 1) return launch_pdl(paged_select_kernel<T, 1>, grid, block, 0, st, c, p, G, NT);
  if (G == 2) return launch_pdl(paged_select_kernel<T, 2>, grid, block, 0, st, c, p, G, NT);
  if (G <= 4) return launch_pdl(paged_select_kernel<T, 4>, grid, block, 0, st, c, p, G, NT);
  return launch_pdl(paged_select_kernel<T, 8>, grid, block, 0, st, c, p, G, NT);
}

template <int NT>
int launch_attend(const PagedView& c, const DecodeP& p, int G, int blocks, cudaStream_t st) {
  const int smem = kStages * (kStageV + ((c.m + 15) & ~15) * TT);
  const int rc = set_smem_limit(paged_attend_kernel<NT>, smem, "paged_attend_kernel");
  if (rc != AQUA_OK) return rc;
  const cudaError_t e = launch_pdl(paged_attend_kernel<NT>, dim3(blocks), dim3(kThreads), smem, st, c, p, G);
  if (e != cudaSuccess) return set_error(AQUA_ERR_CUDA, "paged_attend_kernel: %s", cudaGetErrorString(e));
  return check_launch("paged_attend_kernel");
}

}  // namespace

size_t paged_decode_workspace_bytes(int n_units, int G) { return layout_of(n_units, G, attend_blocks()).total; }

int launch_paged_decode(const PagedView& c, const int32_t* len, const void* q, bool bf16, const Strides& qs,
                        const float* P, const RopeView& rope, int Hq, int k, float scale, void* out, bool out_bf16,
                        int32_t* sel_out, float* qproj_out, float* lse_out, void* ws, cudaStream_t st) {
  const int n_units = c.B * c.Hkv, G = Hq / c.Hkv, NT = G > 4 ? 2 : 1, blocks = attend_blocks();
  const Layout y = layout_of(n_units, G, blocks);
  uint8_t* base = static_cast<uint8_t*>(ws);
  DecodeP p;
  p.len = len; p.q = q; p.qs = qs; p.P = P; p.rope = rope; p.Hq = Hq; p.k = k; p.scale = scale;
  p.out = out; p.out_bf16 = out_bf16; p.sel_out = sel_out; p.qproj_out = qproj_out; p.lse_out = lse_out;
  p.ucount = reinterpret_cast<int32_t*>(base + y.ucount);
  p.ulist = base + y.ulist;
  p.qfrag = reinterpret_cast<uint2*>(base + y.qfrag);
  p.qfac = reinterpret_cast<float*>(base + y.qfac);
  p.part_ml = reinterpret_cast<float2*>(base + y.part_ml);
  p.split = reinterpret_cast<int4*>(base + y.split);
  p.part_o = reinterpret_cast<float*>(base + y.part_o);
  cudaError_t e = bf16 ? launch_select<__nv_bfloat16>(c, p, G, NT, st) : launch_select<float>(c, p, G, NT, st);
  if (e != cudaSuccess) return set_error(AQUA_ERR_CUDA, "paged_select_kernel: %s", cudaGetErrorString(e));
  int rc = check_launch("paged_select_kernel");
  if (rc != AQUA_OK) return rc;
  rc = NT == 1 ? launch_attend<1>(c, p, G, blocks, st) : launch_attend<2>(c, p, G, blocks, st);
  if (rc != AQUA_OK || blocks < 2) return rc;
  e = launch_pdl(paged_merge_kernel, dim3(blocks - 1, G), dim3(kMergeWarps * 32), 0, st, c, p, G);
  if (e != cudaSuccess) return set_error(AQUA_ERR_CUDA, "paged_merge_kernel: %s", cudaGetErrorString(e));
  return check_launch("paged_merge_kernel");
}

}  // namespace aqua
