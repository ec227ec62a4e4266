// One decode step of AQUA attention over the paged 8-bit cache.
//
// paged_select_kernel, a block per KV head g and a few sequences b: for the group's
// query heads q~ = rope(q, len - 1) P (f64, rounded once), the k largest |q~_j|
// (ties to the lower j), the union U of the kept dimensions as a bit mask, and the
// masked queries in the layout the tensor cores take them.
//
// paged_attend_kernel, persistent: the tokens of all (b, g) are cut into tiles
// of 128, the flat sequence of tiles into pieces.  Every block has one piece, with
// five eighths of the work together; the rest are as many smaller pieces that a
// block takes when it is done (equal shares left the slowest block 15 to 20 %
// behind the median).  Short jobs have equal shares only.
//
//   s_t  = ks(page) sum_{j in U} q~_j code_t[j] / sqrt(d)
//   w_t  = s_t log2(e) + log2 vs(page),   p_t = 2^(w_t - M),  M a lazily raised max of w
//   O   += p_t code_t[v],                 l += p_t / vs(page)
//   out  = O / l,   lse = ln2 (M + log2 l)
//
// Taking the value scale into the exponent makes O a plain sum over codes, so
// pages with different scales share one accumulator, and what weighs most in O
// has p near 1.
//
// Both products run on tcgen05 (kind::f8f6f4) straight from the codes: a tile's
// kept key rows [dim][128 tokens] and its value rows [token][128 dims] are each
// the M-major A operand as they lie in the pages, so no code is ever converted.
// The B operands are sums of 8-bit parts.  q~: e4m3, 16 times finer each, four for
// a bf16 output (15 bits or more), six for an f32 one (about 24).  p: e5m2, whose
// five exponent bits are those of f16: four parts for a bf16 output, 8 times finer
// each (2^-12 of p); for an f32 one an f16 number cut into four and what its rounding
// left cut into four more (2^-22).  With 2^12 to 2^15 for the largest p, a weight
// down to 2^-25 of it keeps its bits, and one is lost only below 2^-37 (2^-49): a
// key that outweighs a long tail and has a value of nearly nothing leaves the tail
// its share.  (Three e4m3 parts, a grid of 2^-23 of the largest, lost such a tail
// from 15 nats on.)
// N = parts x heads is 16 to 64 columns; a product of 128 x 128 x N reads 16 KB
// of A, so the columns cost next to nothing.  (Products on mma.sync f16, with
// every code converted in registers, left the kernel bound by instructions: 73 us
// for 131072 tokens x 8 heads against 41 us of memory time.)
//
// Warps 0-3 own one token a thread: scores from tensor memory, softmax, parts of
// p to shared memory.  Warp 4 issues the products.  Warp 5 walks the pieces and
// has the value rows brought by tensor copies, one a page.  Warps 6-9 gather the
// key rows in U (zeros for those no head kept) in 16-byte pieces, 16 tokens of a dim
// each, in the same 128-byte swizzle.  A key buffer is free as soon as its scores
// are, a value buffer only after the softmax and its product, a path of 9000 cycles:
// two key and four value buffers of 16 KB, two blocks an SM.  The first tiles are
// fetched while the selection still runs, with all their key rows.
// A piece that starts or ends inside a (b, g) leaves (M, l, O); paged_merge_kernel
// adds the parts in the order of the tokens, and forms those heads again that a NaN
// key in a dimension they left out made NaN.  Which block took a piece changes
// nothing, so results do not depend on timing.
//
// Measured, three launches replayed from a graph: 131072 tokens x 8 heads 58 us
// (268 MB of rows a head kept: 4.6 TB/s), 32 sequences of up to 32768 tokens, 8
// heads of 8 queries, 194 us (4.9 TB/s), 8 x 8192 tokens 39.5 us; with f32 outputs
// 63, 328 and 44 us.  With up to
// four heads a group the middle of a job is bound by memory (1.5 us a tile and
// block, two blocks an SM), with eight by the softmax warps' chain of a tile; to
// that come 9 us until the selection is done and the first scores are there,
// and 4 us of tail and merge.
//
// edgentiq, "How AQUA Works", Online Inference: scores on the selected
// dimensions, softmax, weighted sum of the unprojected values.
#include <math.h>

#include "paged_internal.cuh"

namespace aqua {

namespace {

constexpr int D = kHeadDim;
constexpr int TT = 128;                    // tokens per tile
constexpr int kSoftThreads = 128;         // one thread per token of a tile
constexpr int kMmaWarp = 4, kValWarp = 5, kKeyWarp0 = 6;
constexpr int kKeyThreads = 128;
constexpr int kThreads = kKeyWarp0 * 32 + kKeyThreads;
constexpr int kVStages = 4, kKStages = 2;
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
  int32_t* ctrl;
  // workspace
  uint4* umask;          // [n_units] the dims any head of the group kept
  uint8_t* qpart;        // [n_units][N][D] e4m3 parts of the masked queries: row h * stride + part
  float* qfac;           // [n_units][kMaxG] factor of a head's scores (log2 domain, without the key scale)
  int32_t* prefix;       // [B + 1] tiles of one KV head before each sequence
  int32_t* ctl;          // [0] pieces taken beyond the first ones, [1] units to merge, [2] heads to form again
  float2* part_ml;       // [2 * pieces][G] (M, l) of a partial result
  float* part_o;         // [2 * pieces][G][D]
  int4* split;           // [pieces] units to merge, in any order: unit .x has its tiles in pieces .y ... .z; .w: slot of
                         // piece .y's part
  int32_t* again;        // [n_units * kMaxG] heads with a NaN that is not their query's: unit * kMaxG + head
};

__device__ __forceinline__ int n_tiles(int len) { return (len + TT - 1) / TT; }

__device__ __forceinline__ int seq_tokens(const PagedView& c, const DecodeP& p, int b) {
  bool bad;
  return checked_len(__ldg(p.len + b), c, p.rope.cs ? p.rope.n_pos : 0x7fffffff, bad);
}

__device__ __forceinline__ void store_out_elem(const DecodeP& p, size_t i, float v) {
  if (p.out_bf16)
    static_cast<__nv_bfloat16*>(p.out)[i] = __float2bfloat16_rn(v);
  else
    static_cast<float*>(p.out)[i] = v;
}

// result of a softmax sum: no visible token gives 0 and -inf, NaN stays
__device__ __forceinline__ float normalised(float O, float L) { return L == 0.f ? 0.f : O / L; }
// (L held times 2^up; taken off the logarithm, since M may be so large that a difference of it would be rounded)
__device__ __forceinline__ float lse_of(float M, float L, float up) { return L == 0.f ? -INFINITY : kLn2 * (M + (log2f(L) - up)); }

// ============================================================================
// rotation, projection, top-k
// ============================================================================

// The projection runs on the f64 matrix instruction, heads as rows (those past G are zeros), eight columns of P a
// warp: on f64 FMAs, every thread a column and all heads, the reads of q~ from shared memory took 5 of 7 us a
// sequence.  What is left is a chain of latencies: P is loaded with the first queries, the next
// sequence's queries during this one's projection, and after it each head is one warp's business.  64 registers
// leave room for an attention block, or a second block of this kernel, beside this one.
__device__ __forceinline__ void mma_f64(double2& d, double a, double b) {
  asm volatile("mma.sync.aligned.m8n8k4.row.col.f64.f64.f64.f64 {%0, %1}, {%2}, {%3}, {%0, %1};"
               : "+d"(d.x), "+d"(d.y)
               : "d"(a), "d"(b));
}

template <typename T>
__global__ void __launch_bounds__(kSelThreads, 2) paged_select_kernel(PagedView c, DecodeP p, int G, int NH, int stride, int parts, int group) {
  static_assert(kSelThreads == 4 * D && kMaxG == 8, "eight columns a warp, eight rows an instruction");
  constexpr int kEach = kMaxG * D / kSelThreads;      // elements of the group's queries a thread
  __shared__ __align__(16) double qd[kMaxG][D + 8];   // rotated rows; the pad keeps the fragments' reads apart
  __shared__ __align__(16) float raw[kMaxG][D], qs[kMaxG][D];
  __shared__ uint32_t kept[kMaxG][4];
  __shared__ int before;
  const int g = blockIdx.y;
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  // fragment of the instruction: row (head) or column lane / 4; input dims 8 s + 2 (lane % 4), + 1 for step 2 s, 2 s + 1
  const int fr = lane >> 2, fk = 2 * (lane & 3);
  prefetch_head(p.P + (size_t)g * D * D, tid, kSelThreads);
  for (int i = tid; i < kMaxG * (D + 8); i += kSelThreads) qd[0][i] = 0.0;
  pdl_wait();
  pdl_launch_dependents();
  if (tid == 0 && blockIdx.x == 0 && g == 0) p.ctl[0] = p.ctl[1] = p.ctl[2] = 0;
  const int b_end = min(c.B, ((int)blockIdx.x + 1) * group);
  int len = 0;
  T x[kEach];                               // as it lies in memory: a conversion here would wait for the load
  auto fetch = [&](int b) {
    len = __ldg(p.len + b);
    const T* q = static_cast<const T*>(p.q) + (size_t)b * p.qs.row + (size_t)g * G * p.qs.head;
#pragma unroll
    for (int y = 0; y < kEach; ++y) {
      const int i = tid + y * kSelThreads;
      if ((i >> 7) < G) x[y] = q[(size_t)(i >> 7) * p.qs.head + (i & 127)];
    }
  };
  fetch(blockIdx.x * group);
  float pr[D / 4];
  {
    const float* Pg = p.P + (size_t)g * D * D + (size_t)fk * D + 8 * w + fr;
#pragma unroll
    for (int i = 0; i < D / 4; i += 2) {
      pr[i] = __ldg(Pg + 4 * i * D);
      pr[i + 1] = __ldg(Pg + 4 * i * D + D);
    }
  }
#pragma unroll 1
  for (int b = blockIdx.x * group; b < b_end; ++b) {
    const int u = b * c.Hkv + g;
    bool bad;
    const int n = checked_len(len, c, p.rope.cs ? p.rope.n_pos : 0x7fffffff, bad);
    const bool turn = p.rope.cs != nullptr && n > 0;
    if (turn) {
#pragma unroll
      for (int y = 0; y < kEach; ++y) raw[(tid + y * kSelThreads) >> 7][tid & 127] = (float)x[y];
    }
    if (tid == 0) {
      if (bad) report_arg(c);
      before = 0;
    }
    __syncthreads();
    const float* cs = p.rope.cs + (size_t)(n - 1) * p.rope.rot;
#pragma unroll
    for (int y = 0; y < kEach; ++y) {
      const int hh = (tid + y * kSelThreads) >> 7, j = tid & 127;
      if (hh < G) qd[hh][j] = turn ? rotated<double>(raw[hh], j, cs, p.rope.rot, p.rope.interleaved) : (double)(float)x[y];
    }
    __syncthreads();
    if (b + 1 < b_end) fetch(b + 1);
    {
      double2 even = make_double2(0.0, 0.0), odd = make_double2(0.0, 0.0);
#pragma unroll
      for (int i = 0; i < D / 4; i += 2) {
        const double2 a = *reinterpret_cast<const double2*>(&qd[fr][4 * i + fk]);
        mma_f64(even, a.x, (double)pr[i]);
        mma_f64(odd, a.y, (double)pr[i + 1]);
      }
      // row fr, columns 8 w + fk, + 1
      *reinterpret_cast<float2*>(&qs[fr][8 * w + fk]) = make_float2((float)(even.x + odd.x), (float)(even.y + odd.y));
    }
    __syncthreads();
    if (w < G) {
      // ---- head w: lane holds dims lane + 32 y
      float qt[4];
      uint32_t key[4];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int i = lane + 32 * y;
        qt[y] = qs[w][i];
        // magnitude order as unsigned order; dims past d_store below every candidate, NaN payloads one key
        key[y] = i < c.m ? min(__float_as_uint(fabsf(qt[y])), 0x7F800001u) + 1u : 0u;
        if (p.qproj_out) p.qproj_out[((size_t)b * p.Hq + (size_t)g * G + w) * D + i] = qt[y];
      }
      // tau: the largest value with at least k keys >= tau, two bits a round from the top, the three counts in one
      // word; the search ends when exactly k are
      uint32_t tau = 0;
      int cnt = D;
#pragma unroll 1
      for (int bit = 30; bit >= 0 && cnt != p.k; bit -= 2) {
        const uint32_t c1 = tau | (1u << bit), c2 = tau | (2u << bit), c3 = tau | (3u << bit);
        uint32_t n = 0;
#pragma unroll
        for (int y = 0; y < 4; ++y) n += (key[y] >= c1 ? 1u : 0u) + (key[y] >= c2 ? 0x100u : 0u) + (key[y] >= c3 ? 0x10000u : 0u);
        n = __reduce_add_sync(0xffffffffu, n);         // each at most 128
        const int n1 = n & 255, n2 = (n >> 8) & 255, n3 = n >> 16;
        if (n1 >= p.k) {
          tau = n3 >= p.k ? c3 : n2 >= p.k ? c2 : c1;
          cnt = n3 >= p.k ? n3 : n2 >= p.k ? n2 : n1;
        }
      }
      uint32_t word[4];
#pragma unroll
      for (int y = 0; y < 4; ++y) word[y] = __ballot_sync(0xffffffffu, key[y] >= tau && key[y] > 0);
      if (cnt != p.k) {
        // equal keys straddle the cut: every key above tau, then keys equal to tau from the lowest dim up
        int need = p.k;
#pragma unroll
        for (int y = 0; y < 4; ++y) need -= __popc(__ballot_sync(0xffffffffu, key[y] > tau));
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const uint32_t eq = __ballot_sync(0xffffffffu, key[y] == tau && key[y] > 0);
          const bool take = key[y] > tau || (key[y] == tau && key[y] > 0 && __popc(eq & ((1u << lane) - 1u)) < need);
          need -= min(need, __popc(eq));
          word[y] = __ballot_sync(0xffffffffu, take);
        }
      }
      float mx = 0.f;
      int pos = 0;
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const bool keep = (word[y] >> lane) & 1u;
        if (keep) {
          if (p.sel_out)
            p.sel_out[((size_t)b * p.Hq + (size_t)g * G + w) * p.k + pos + __popc(word[y] & ((1u << lane) - 1u))] = lane + 32 * y;
          mx = fmaxf(mx, finite_abs(qt[y]));
        } else {
          qt[y] = 0.f;
        }
        pos += __popc(word[y]);
        if (lane == 0) kept[w][y] = word[y];
      }
      mx = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mx)));
      // 2^(7-e) with mx = f 2^e brings the largest entry to [128, 256): e4m3 reaches 448 and 2^-9.  Any finite entry
      // has e <= 127; from below 2^-116 on entries get smaller than that, but keep the factor a normal number.
      const int e = max((int)(__float_as_uint(mx) >> 23) - 127, -116);
      const float mul = __uint_as_float((uint32_t)(127 + 7 - e) << 23);
      // parts: x = x0 + x1 / 16 + x2 / 256 + ..., each the e4m3 number nearest to what is left (a remainder is at
      // most half a step, so 16 times it stays in range)
      uint8_t* dst = p.qpart + ((size_t)u * NH + w) * stride * D + lane;
      bool lost = false;
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        qt[y] *= mul;
        if (!(fabsf(qt[y]) < INFINITY)) {              // an infinite query makes its scores NaN, not the largest code
          qt[y] = NAN;
          lost = true;
        }
      }
      lost = __any_sync(0xffffffffu, lost);
      if (lane == 0)
        p.qfac[(size_t)u * kMaxG + w] = lost ? NAN : __uint_as_float((uint32_t)(127 - 7 + e) << 23) * p.scale * kLog2e;
#pragma unroll 1
      for (int i = 0; i < stride; ++i, dst += D) {
        const uint32_t code = i < parts ? f32x4_to_e4m3x4(qt[0], qt[1], qt[2], qt[3]) : 0u;
        const float2 b0 = e4m3x2_to_f32x2((uint16_t)code), b1 = e4m3x2_to_f32x2((uint16_t)(code >> 16));
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const uint8_t byte = (uint8_t)(code >> (8 * y));
          // the first part of a kept entry is never +0, which marks those that are left out
          dst[32 * y] = i == 0 && byte == 0 && ((word[y] >> lane) & 1u) ? 0x80 : byte;
        }
        qt[0] = (qt[0] - b0.x) * 16.f;
        qt[1] = (qt[1] - b0.y) * 16.f;
        qt[2] = (qt[2] - b1.x) * 16.f;
        qt[3] = (qt[3] - b1.y) * 16.f;
      }
    } else if (w >= 8) {
      // zeros for the heads the operand has room for but the group lacks
      for (int i = tid - 256; i < (NH - G) * stride * (D / 16); i += kSelThreads - 256)
        reinterpret_cast<uint4*>(p.qpart + ((size_t)u * NH + G) * stride * D)[i] = make_uint4(0, 0, 0, 0);
      // tiles of the sequences before this one (one block of each sequence)
      if (g == 0) {
        int sum = 0;
        for (int x = tid - 256; x < b; x += kSelThreads - 256) sum += n_tiles(seq_tokens(c, p, x));
        sum = __reduce_add_sync(0xffffffffu, sum);
        if (lane == 0 && sum != 0) atomicAdd(&before, sum);
      }
    }
    __syncthreads();
    if (tid == 0) {
      uint4 um = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int hh = 0; hh < kMaxG; ++hh) {
        if (hh >= G) break;
        um.x |= kept[hh][0];
        um.y |= kept[hh][1];
        um.z |= kept[hh][2];
        um.w |= kept[hh][3];
      }
      p.umask[u] = um;
      if (g == 0) {
        p.prefix[b] = before;
        if (b == c.B - 1) p.prefix[c.B] = before + n_tiles(n);
      }
    }
    // an empty sequence has no tiles: attention over no token is 0 with lse -inf
    if (n == 0) {
      const size_t r0 = (size_t)b * p.Hq + (size_t)g * G;
      for (int i = tid; i < G * D; i += kSelThreads) store_out_elem(p, r0 * D + i, 0.f);
      if (p.lse_out && tid < G) p.lse_out[r0 + tid] = -INFINITY;
    }
    __syncthreads();
  }
}

// ============================================================================
// attention
// ============================================================================

constexpr int kStageV = D * TT;                       // bytes of a tile's value rows

// Position in the flat sequence of tiles.
struct Cursor {
  int u;                   // unit (b * Hkv + g)
  int b, g;
  int len;                 // tokens of the sequence
  int tile;                // tile of the unit
};

// a / b for a, b >= 0: a division of 64 bits takes several hundred cycles, one of 32 bits some tens
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// The flat sequence of `total` tiles as pieces: nb first ones, then smaller ones.
struct Pieces {
  long long total, nb;
  long long first, rest;   // tiles of a first piece and of a later one; first = 0: equal shares, nothing else
  __device__ __forceinline__ Pieces(long long t, int blocks) : total(t), nb(min((long long)blocks, t)), first(0), rest(1) {
    // worth it from five tiles a block on: one later piece each (three took 59.7 us in place of 54.0 for 8192 tiles of
    // 8 heads, a change of pieces costs 2 us; none: 52, but 216 in place of 189 for the 43000 of 32 sequences)
    if (nb > 0 && total >= 5 * nb) {
      first = total * 5 / 8 / nb;
      rest = (total - first * nb + nb - 1) / nb;
    }
  }
  __device__ __forceinline__ long long start(long long p) const {
    if (first == 0) return p * total / nb;
    return p <= nb ? p * first : min(total, nb * first + (p - nb) * rest);
  }
  __device__ __forceinline__ int of(long long tile) const {
    if (first == 0) return (int)(((tile + 1) * nb - 1) / total);
    return (int)(tile < nb * first ? quotient(tile, first) : nb + quotient(tile - nb * first, rest));
  }
  __device__ __forceinline__ int count() const {
    return (int)(first == 0 ? nb : nb + (total - nb * first + rest - 1) / rest);
  }
};

// What a tile is: written by the value warp when it issues its copies.
struct TileInfo {
  int b, g, u, len, tile;
  int slot;                // where the piece's part of this unit goes; < 0: the piece has the whole unit
  int q;                   // buffer with the unit's queries
  int flags;
};
enum TileFlag { kFirst = 1, kLast = 2, kEnd = 4,     // of the piece's part of a unit; of the block's work
                kFresh = 8 };                        // O starts from zero

struct AttendMisc {
  uint64_t known[kVStages];                 // a tile's info is written
  uint64_t v_full[kVStages], v_empty[kVStages];   // value rows landed / their product is done
  uint64_t k_full[kKStages], k_empty[kKStages];   // key rows, scales and queries landed / the scores are done
  uint64_t s_full[2], p_full[2], pv_done[2];
  uint64_t drain;
  TileInfo info[kVStages];
  int pid[kVStages][TT / 16];      // its pages, one every 16 tokens; -1: none
  int stop[2];                     // softmax threads leave after this (even, odd) tile
  float ks[kVStages][TT / 16];     // key scale of every 16 tokens; negative: their page does not exist
  float vs[kVStages][TT / 16];
  float fac[kVStages][kMaxG];      // factors of a unit's queries, at its first tile
  union {
    float red[4][kMaxG];
    long long scan[kThreads / 32];          // before the roles begin
  };
  Cursor cur;
  uint32_t tmem;
  int abort;
};

static_assert(sizeof(AttendMisc) <= 1024, "two blocks an SM: 113 KB each, 112 of them tiles and operands");

__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// the box of the map from row y on, to shared memory
__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap* map, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(y), "r"(smem_u32(bar))
      : "memory");
}

// ------------------------------------------------------------------ tcgen05 wrappers
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
// D[tmem] (+)= A[smem] * B[smem], 8-bit floats in, f32 accumulate
__device__ __forceinline__ void tc_mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}
// 16 consecutive f32 columns of this warp's 32 TMEM lanes
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float* v) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(taddr),
      "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3])),
      "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])), "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7])),
      "r"(__float_as_uint(v[8])), "r"(__float_as_uint(v[9])), "r"(__float_as_uint(v[10])),
      "r"(__float_as_uint(v[11])), "r"(__float_as_uint(v[12])), "r"(__float_as_uint(v[13])),
      "r"(__float_as_uint(v[14])), "r"(__float_as_uint(v[15]))
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory matrix descriptor, 128-byte swizzle, one swizzle atom wide: groups of eight rows of 128
// bytes, 1024 bytes apart.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFF) | ((uint64_t)(1024 >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}
// kind::f8f6f4: e4m3 A (M-major), e4m3 or e5m2 B (K-major), f32 D, 128 x N
enum Fp8Type { kE4m3 = 0, kE5m2 = 1 };
__host__ __device__ constexpr uint32_t idesc_f8(int N, Fp8Type b) {
  return (1u << 4) | ((uint32_t)b << 10) | (1u << 15) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(TT >> 4) << 24);
}

// Bounded wait that gives up at once when another role did; the first to give up reports.  The value warp and
// the softmax threads go on to a point where all of them leave (every later wait returns at once), so that
// no barrier among them is left waiting; what they write then is garbage, in bounds.
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, volatile int* abort, int32_t* ctrl) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = globaltimer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*abort) return false;
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      *abort = 1;
      record_status(ctrl, AQUA_ERR_TIMEOUT);
      return false;
    }
  }
}

__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// For a polling loop that began at time `since` (0: sets it): whether to give up.
__device__ __forceinline__ bool poll_abort(volatile int* abort, unsigned long long& since, int32_t* ctrl) {
  const unsigned long long now = globaltimer_ns();
  if (since == 0) since = now;
  if (*abort) return true;
  if (now - since <= kWaitLimitNs) return false;
  *abort = 1;
  record_status(ctrl, AQUA_ERR_TIMEOUT);
  return true;
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
__device__ __forceinline__ void next_tile(const PagedView& c, const DecodeP& p, Cursor& cur) {
  if (++cur.tile >= n_tiles(cur.len)) next_unit(c, p, cur);
}

constexpr float kLazy = 3.f;        // the reference M is raised when a score exceeds it by 2^3
constexpr float kPScale = 12.f;     // p is held times 2^12: at most 2^15, below the largest f16 and e5m2 numbers

// The tensor cores cut each sum they extend off, always towards zero: over the thousands of extensions that a long
// unit has in one block the losses add up (2e-4 of the output after 3000 tiles).  For f32 outputs O goes to registers
// every kFlush tiles, 64 extensions: at most 64 / 2 steps of 2^-23, 4e-6.  l does the same in each thread, so that
// small weights are added to each other before they meet a large one (1.2e-5 off after 256 tiles otherwise).  A bf16 output's rounding covers 2^-10, four thousand tiles of a unit in a block.
constexpr int kFlush = 16;

// 8 (a - b) of two pairs, exact where a and b are close
__device__ __forceinline__ float2 eight_times(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, e, n;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 e, {%6, %6};\n\tmov.b64 n, {%7, %7};\n\t"
      "mul.rn.f32x2 x, x, e;\n\tfma.rn.f32x2 x, y, n, x;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(8.f), "f"(-8.f));
  return r;
}

// the four columns of p's f16 number, each part 8 times finer than the one before
__device__ __forceinline__ float join_p(const float* v) {
  return fmaf(fmaf(fmaf(v[3], 0.125f, v[2]), 0.125f, v[1]), 0.125f, v[0]);
}

// Columns of the B operands: head h, part i in column STR h + i; NH heads.
template <int STR, int NH>
struct Cols {
  static constexpr int N = STR * NH;
  static constexpr int QPARTS = STR == 4 ? 4 : 6;
  static constexpr int PPARTS = STR;       // four of an f16 number, or of two
  static constexpr int TMEM = N <= 16 ? 64 : (N <= 32 ? 128 : 256);   // S(even), S(odd), O
  static constexpr int CTAS = N <= 32 ? 2 : 1;                        // blocks an SM (shared memory)
  static __host__ __device__ int smem(int m) {
    return kVStages * kStageV + kKStages * ((m + 31) & ~31) * TT + 4 * N * TT + (int)sizeof(AttendMisc);
  }
};

template <int STR, int NH>
__global__ void __launch_bounds__(kThreads, (Cols<STR, NH>::CTAS)) paged_attend_kernel(const __grid_constant__ CUtensorMap vmap, PagedView c, DecodeP p, int G) {
  using CC = Cols<STR, NH>;
  constexpr int N = CC::N;
  extern __shared__ __align__(1024) uint8_t dyn[];
  const int mrows = (c.m + 31) & ~31;                         // key rows of a tile, zeros past d_store
  const int off_k = kVStages * kStageV, off_q = off_k + kKStages * mrows * TT, off_p = off_q + 2 * N * TT;
  AttendMisc& ms = *reinterpret_cast<AttendMisc*>(dyn + off_p + 2 * N * TT);
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  const uint32_t smem0 = smem_u32(dyn);

  // ---- the tiles, and the unit that this block's first piece starts in (the lengths were written before the
  // selection kernel started, which released this one after its own wait; so were the pages and the table)
  long long total = 0;
  for (int base = 0; base < c.B; base += kThreads) {
    const int b = base + tid;
    const int x = __reduce_add_sync(0xffffffffu, b < c.B ? n_tiles(seq_tokens(c, p, b)) : 0);
    __syncthreads();
    if (lane == 0) ms.scan[w] = x;
    __syncthreads();
    for (int y = 0; y < kThreads / 32; ++y) total += ms.scan[y];
  }
  const Pieces pieces(total * c.Hkv, gridDim.x);
  if (blockIdx.x >= pieces.nb) {
    // The merge waits for this grid alone: with no tokens at all, where every block leaves here, only this wait
    // orders it and what comes after it behind the selection (its counts, its zeros in out).
    pdl_wait();
    return;
  }
  {
    const long long t0 = pieces.start(blockIdx.x);
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
      if (lane == 31) ms.scan[w] = sum;
      __syncthreads();
      long long off = before, all = 0;
      for (int y = 0; y < kThreads / 32; ++y) {
        if (y < w) off += ms.scan[y];
        all += ms.scan[y];
      }
      const long long first = (off + sum - x) * c.Hkv, last = (off + sum) * c.Hkv;
      if (x > 0 && t0 >= first && t0 < last) {
        const int r = (int)(t0 - first);
        ms.cur.b = b;
        ms.cur.g = r / x;
        ms.cur.tile = r % x;
        ms.cur.u = b * c.Hkv + r / x;
        ms.cur.len = len;
      }
      before += all;
    }
  }
  // ---- barriers, tensor memory, the columns of p that no head or part uses (zeros for good)
  if (tid == 0) {
    for (int i = 0; i < kVStages; ++i) {
      mbar_init(&ms.known[i], 1);
      mbar_init(&ms.v_full[i], 1);
      mbar_init(&ms.v_empty[i], 1);
    }
    for (int i = 0; i < kKStages; ++i) {
      mbar_init(&ms.k_full[i], 2 * kKeyThreads);    // every thread's own stores, and its copies
      mbar_init(&ms.k_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ms.s_full[i], 1);
      mbar_init(&ms.p_full[i], kSoftThreads);
      mbar_init(&ms.pv_done[i], 1);
    }
    mbar_init(&ms.drain, 1);
    fence_barrier_init();
    ms.abort = 0;
    for (int i = 0; i < kVStages; ++i) ms.info[i] = TileInfo{0, 0, 0, 0, 0, 0, 0, 0};
  }
  if (w == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&ms.tmem)),
                 "r"((uint32_t)CC::TMEM)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    tc_fence_before();
  }
  for (int i = tid; i < 2 * N * TT / 16; i += kThreads)
    *reinterpret_cast<uint4*>(dyn + off_p + 16 * i) = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ms.tmem;

  // pages of the 512 tokens from a tile on, 16 tokens a lane
  auto page_of_chunk = [&](int b, int tile, int len) {
    int pid = -1;
    const int t = tile * TT + 16 * lane;
    if (t < len) {
      pid = __ldg(c.table + (size_t)b * c.max_pages + (t >> c.page_log2));
      if (pid < 0 || pid >= c.n_pages) {
        pid = -1;
        report_arg(c);
      }
    }
    return pid;
  };
  const int pmask = (1 << c.page_log2) - 1;

  if (w >= kKeyWarp0) {
    // ================= key rows, scales, queries =================
    const int ct = tid - kKeyWarp0 * 32, lc = ct & 7, lr = ct >> 3;    // chunk of 16 tokens, first row (dim)
    auto copy_keys = [&](int t, const TileInfo& ti, const uint4& um) {
      const uint32_t kbase = smem0 + off_k + (t % kKStages) * mrows * TT;
      const int pid = ms.pid[t % kVStages][lc];
      // rows lr, lr + 16, ...; rows that are not wanted are zeros
      const uint8_t* kb = c.k;
      if (pid >= 0) kb += c.kblock(pid, ti.g) + ((ti.tile * TT + 16 * lc) & pmask) + ((size_t)lr << c.page_log2);
      const uint32_t words[4] = {um.x >> lr, um.y >> lr, um.z >> lr, um.w >> lr};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (16 * i >= mrows) break;
        const int r = lr + 16 * i;
        const bool in = pid >= 0 && ((words[i >> 1] >> (16 * (i & 1))) & 1u);
        cp_async16_zfill(kbase + r * TT + ((lc ^ (r & 7)) << 4), kb + (in ? (size_t)(16 * i) << c.page_log2 : 0), in);
      }
      if (ct < TT / 16) {                     // scales of the tile's pages; lc == ct here
        const int st = t % kVStages;
        if (pid >= 0) {
          const size_t si = (size_t)pid * c.Hkv + ti.g;
          cp_async_small<4>(&ms.ks[st][ct], c.ks + si);
          cp_async_small<4>(&ms.vs[st][ct], c.vs + si);
        } else {
          ms.ks[st][ct] = -1.f;
          ms.vs[st][ct] = 1.f;
        }
      }
    };
    auto finish = [&](int t, const TileInfo& ti) {
      if (ti.flags & kFirst) {
        // two tiles ago the buffer's last unit was done with its scores: so this tile's key buffer could be free
        const uint32_t qbase = smem0 + off_q + ti.q * N * TT;
        for (int i = ct; i < N * 8; i += kKeyThreads) {
          const int r = i >> 3, ch = i & 7;
          cp_async16_zfill(qbase + r * D + ((ch ^ (r & 7)) << 4), p.qpart + ((size_t)ti.u * N + r) * D + ch * 16, true);
        }
        // (a tile's slot, not the unit's: the softmax has read it when the tile's value buffer is free again)
        if (ct < G) cp_async_small<4>(&ms.fac[t % kVStages][ct], p.qfac + (size_t)ti.u * kMaxG + ct);
      }
      // the copies arrive when they have landed; the product warp makes them visible to the tensor cores
      cp_async_arrive_noinc(&ms.k_full[t % kKStages]);
      mbar_arrive(&ms.k_full[t % kKStages]);
    };
    auto info_of = [&](int t) {
      wait_or_abort(&ms.known[t % kVStages], (t / kVStages) & 1, &ms.abort, p.ctrl);
      __syncwarp();
      return ms.info[t % kVStages];
    };
    // the first tiles, while the selection runs: all their key rows
    const uint32_t f = 0xffffffffu;
    auto low = [&](int wd) { return c.m >= 32 * wd + 32 ? f : (c.m > 32 * wd ? (1u << (c.m - 32 * wd)) - 1u : 0u); };
    const uint4 all = make_uint4(low(0), low(1), low(2), low(3));
    TileInfo ti = info_of(0);
    copy_keys(0, ti, all);
    const bool two = !(ti.flags & kEnd);
    TileInfo tn = ti;
    if (two) {
      tn = info_of(1);
      copy_keys(1, tn, all);
    }
    pdl_wait();                               // the selection's results
    finish(0, ti);
    if (two) finish(1, tn);
    int iu = -1;
    uint4 um = all;
    for (int t = 2; two && !(tn.flags & kEnd); ++t) {
      tn = info_of(t);
      if (__any_sync(0xffffffffu, *(volatile int*)&ms.abort)) break;      // (no barrier among these warps)
      if (tn.u != iu) {
        iu = tn.u;
        um = p.umask[iu];
      }
      wait_or_abort(&ms.k_empty[t % kKStages], ((t / kKStages) - 1) & 1, &ms.abort, p.ctrl);
      __syncwarp();
      copy_keys(t, tn, um);
      finish(t, tn);
    }
    cp_async_wait_all();
  } else if (w == kValWarp) {
    // ================= pieces, value rows =================
    if (lane == 0) prefetch_tmap(&vmap);
    Cursor cur = ms.cur;
    int piece = blockIdx.x;
    long long begin = pieces.start(piece), stop_at = pieces.start(piece + 1);   // the piece's tiles
    int left = (int)(stop_at - begin);
    const bool more = pieces.first > 0;        // there are later pieces to take
    int iu = -1, ord = -1;
    bool part_first = true, waited = false;    // the piece's first tile is next; the earlier kernels' results may be read
    int seg_first = 0;                         // first tile of the unit in this piece
    int4 split = make_int4(0, 0, 0, 0);
    int split_at = -1;
    // A piece that is the second of a unit's pieces puts the unit on the list of the merge.
    auto note_split = [&]() {
      if (cur.tile == 0) return;
      const long long f = begin - cur.tile;                   // the unit's tiles are [f, f + n)
      const int first = pieces.of(f);
      if (first != piece - 1) return;
      split = make_int4(cur.u, first, pieces.of(f + n_tiles(cur.len) - 1), pieces.start(first) < f ? 1 : 0);
      split_at = atomicAdd(p.ctl + 1, 1);
    };
    // (the entry is stored a little later, when its place is known without a wait)
    auto store_split = [&]() {
      if (split_at >= 0) p.split[split_at] = split;
      split_at = -1;
    };
    // The first value rows come while the selection runs; then its results, and the merge of an earlier call, which
    // has read its parts.
    auto after_wait = [&]() {
      waited = true;
      pdl_wait();
      pdl_launch_dependents();
      if (lane == 0) {
        const Cursor now = cur;
        cur = ms.cur;                          // the first piece's start
        note_split();
        cur = now;
      }
    };
    int next_piece = -1;
    // pages of the four tiles from `base` of unit `base_u` on, eight lanes a tile
    int base = cur.tile, base_u = cur.u, pids = page_of_chunk(cur.b, cur.tile, cur.len);
    for (int t = 0;; ++t) {
      const int st = t % kVStages;
      if (!waited && (t >= kVStages || (more && left <= 3))) after_wait();
      if (t >= kVStages) wait_or_abort(&ms.v_empty[st], ((t / kVStages) - 1) & 1, &ms.abort, p.ctrl);
      __syncwarp();
      // the piece after this one: asked for a few tiles before the end, needed at the last tile
      if (left == 3 || (part_first && left < 3)) {
        next_piece = -1;
        if (lane == 0 && more && !*(volatile int*)&ms.abort) next_piece = (int)pieces.nb + atomicAdd(p.ctl, 1);
      }
      if (left == 1) {
        next_piece = __shfl_sync(0xffffffffu, next_piece, 0);
        if (next_piece >= pieces.count()) next_piece = -1;
      }
      const bool change = cur.u != iu || part_first, end = left == 1 && next_piece < 0;
      if (change) {
        iu = cur.u;
        ++ord;
        part_first = false;
        seg_first = cur.tile;
      }
      int mypid = __shfl_sync(0xffffffffu, pids, 8 * (cur.tile - base) + (lane & 7));
      if (lane >= TT / 16) mypid = -1;
      if (lane < TT / 16) ms.pid[st][lane] = mypid;
      __syncwarp();
      if (lane == 0) {
        const bool unit_end = cur.tile + 1 == n_tiles(cur.len);
        TileInfo ti;
        ti.b = cur.b; ti.g = cur.g; ti.u = cur.u; ti.len = cur.len; ti.tile = cur.tile;
        // a part that does not start the piece is its second
        ti.slot = unit_end && seg_first == 0 ? -1 : 2 * piece + (begin + (cur.tile - seg_first) < stop_at - left ? 1 : 0);
        ti.q = ord & 1;
        ti.flags = (change ? kFirst : 0) | (change || (STR == 8 && (cur.tile - seg_first) % kFlush == 0) ? kFresh : 0) | (unit_end || left == 1 ? kLast : 0) | (end ? kEnd : 0);
        ms.info[st] = ti;
        mbar_arrive(&ms.known[st]);
      }
      // one copy for each page with tokens (rows of the tile past the length, or without a page, hold what they
      // held; the softmax threads zero them)
      const bool go = mypid >= 0 && ((cur.tile * TT + 16 * lane) & pmask) == 0;
      const uint32_t n_go = __popc(__ballot_sync(0xffffffffu, go));
      if (lane == 0) mbar_arrive_expect_tx(&ms.v_full[st], n_go * (uint32_t)(D << c.page_log2));
      __syncwarp();
      if (go)
        tma_rows(smem0 + st * kStageV + 16 * lane * D, &vmap, (mypid * c.Hkv + cur.g) << c.page_log2, &ms.v_full[st]);
      store_split();
      if (end) break;
      if (--left > 0) {
        next_tile(c, p, cur);
      } else {
        // the first tile of the next piece: its sequence by the tiles before each one, 32 probes at a time
        piece = next_piece;
        begin = pieces.start(piece);
        stop_at = pieces.start(piece + 1);
        left = (int)(stop_at - begin);
        const int want = (int)quotient(begin, c.Hkv);
        int lo = 0, hi = c.B, before, len;     // prefix[lo] <= want < prefix[hi]
        do {
          const int step = (hi - lo + 31) / 32, at = lo + lane * step;
          const int tiles = at < hi ? __ldcg(p.prefix + at) : 0x7fffffff, tokens = at < hi ? seq_tokens(c, p, at) : 0;
          const int k = 31 - __clz(__ballot_sync(0xffffffffu, at < hi && tiles <= want));   // lane 0 is always under
          before = __shfl_sync(0xffffffffu, tiles, k);
          len = __shfl_sync(0xffffffffu, tokens, k);
          hi = min(hi, lo + (k + 1) * step);
          lo += k * step;
        } while (hi - lo > 1);
        // sequences without tiles share their prefix with the next one: lo is the last of them, which has tiles
        cur.b = lo;
        cur.len = len;
        const int x = n_tiles(len), r = (int)(begin - (long long)before * c.Hkv);
        cur.g = r / x;
        cur.tile = r % x;
        cur.u = lo * c.Hkv + cur.g;
        part_first = true;
      }
      if (cur.u != base_u || (unsigned)(cur.tile - base) >= 4u) {
        base = cur.tile;
        base_u = cur.u;
        pids = page_of_chunk(cur.b, cur.tile, cur.len);
      }
      if (part_first && lane == 0) note_split();
    }
    if (!waited) after_wait();
    store_split();
  } else if (w == kMmaWarp) {
    // ================= products =================
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_f8(N, kE4m3), idesc_p = idesc_f8(N, kE5m2);
      uint32_t fresh = 0;                     // bit t & 31: O starts from zero with tile t
      int n_all = 0x7fffffff;                 // tiles, once known
      bool ok = true;
      auto issue_s = [&](int t) {
        const int fl = ms.info[t % kVStages].flags;
        fresh = (fresh & ~(1u << (t & 31))) | ((fl & kFresh ? 1u : 0u) << (t & 31));
        if (fl & kEnd) n_all = t + 1;
        fence_proxy_async_smem();
        tc_fence_after();
        const uint64_t ad = smem_desc(smem0 + off_k + (t % kKStages) * mrows * TT);
        const uint64_t bd = smem_desc(smem0 + off_q + ms.info[t % kVStages].q * N * TT);
#pragma unroll
        for (int k = 0; k < D / 32; ++k)      // 32 dims: 32 rows of A, 32 bytes of B's rows
          if (32 * k < mrows) tc_mma_f8(tmem + (t & 1) * N, ad + k * (32 * TT >> 4), bd + k * 2, idesc, k > 0);
        tc_commit(&ms.s_full[t & 1]);
        tc_commit(&ms.k_empty[t % kKStages]);
      };
      // Whatever is ready first: the scores of tile t + 1 (its copies landed; its buffer was read before p(t - 1)
      // was announced) or the values of tile t (p written).  In a fixed order either one would hold up the other.
      int scored = 0;                         // tiles whose scores are issued
      for (int t = 0; ok && t < n_all; ++t) {
        unsigned long long since = 0;
        while (true) {
          if (scored < n_all && scored <= t + 1 && mbar_test(&ms.k_full[scored % kKStages], (scored / kKStages) & 1))
            issue_s(scored++);
          if (scored > t && mbar_test(&ms.p_full[t & 1], (t >> 1) & 1) &&
              mbar_test(&ms.v_full[t % kVStages], (t / kVStages) & 1))
            break;
          if (poll_abort(&ms.abort, since, p.ctrl)) {
            ok = false;
            break;
          }
        }
        if (!ok) break;
        fence_proxy_async_smem();
        tc_fence_after();
        const uint64_t ad = smem_desc(smem0 + (t % kVStages) * kStageV);
        const uint64_t bd = smem_desc(smem0 + off_p + (t & 1) * N * TT);
        const bool first = (fresh >> (t & 31)) & 1u;
#pragma unroll
        for (int k = 0; k < TT / 32; ++k)
          tc_mma_f8(tmem + 2 * N, ad + k * (32 * D >> 4), bd + k * 2, idesc_p, k > 0 || !first);
        tc_commit(&ms.pv_done[t & 1]);
        tc_commit(&ms.v_empty[t % kVStages]);
      }
      tc_commit(&ms.drain);                   // nothing is in flight when tensor memory is given back
      mbar_wait_bounded(&ms.drain, 0);
    }
    __syncwarp();
  } else {
    // ================= softmax: thread = token of the tile, and dim of the output =================
    pdl_wait();
    const uint32_t lane_base = tmem + ((uint32_t)(32 * w) << 16);
    float fac[NH], ref[NH], l[NH];
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      wait_or_abort(bar, parity, &ms.abort, p.ctrl);
      __syncwarp();                           // what follows is executed by whole warps
    };
    // this thread's byte in row n of p: chunk (tid / 16) ^ (n % 8)
    const uint32_t pcol = (uint32_t)(tid & 15);
    const uint32_t pchunk = (uint32_t)(tid >> 4);
    bool begun = false;                       // O holds tiles of this part
    float acc[STR == 8 ? NH : 1], lacc[STR == 8 ? NH : 1];      // what it held before it started afresh, and l likewise
    // O of head h of the sixteen columns v, from column cb on
    auto head_of = [&](const float* v, int hl) {
      const float O = join_p(v + hl * STR);
      return STR == 8 ? fmaf(join_p(v + hl * STR + 4), 1.f / 4096.f, O) : O;
    };
    for (int t = 0;; ++t) {
      const int st = t % kVStages, buf = t & 1;
      wait(&ms.known[st], (t / kVStages) & 1);
      const TileInfo ti = ms.info[st];
      if (ti.flags & kFirst) {
        begun = false;
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          ref[h] = -INFINITY;
          l[h] = 0.f;
          if (STR == 8) acc[h] = lacc[h] = 0.f;
        }
      } else if (STR == 8 && (ti.flags & kFresh)) {
        wait(&ms.pv_done[(t - 1) & 1], ((t - 1) >> 1) & 1);
        tc_fence_after();
#pragma unroll
        for (int cb = 0; cb < N; cb += 16) {
          float v[16];
          tmem_ld16(lane_base + 2 * N + cb, v);
          tmem_wait_ld();
#pragma unroll
          for (int hl = 0; hl < 16 / STR; ++hl) acc[cb / STR + hl] += head_of(v, hl);
        }
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          lacc[h] += l[h];
          l[h] = 0.f;
        }
        begun = false;
      }
      wait(&ms.s_full[buf], (t >> 1) & 1);    // and the scales have landed, before the scores were issued
      tc_fence_after();
      if (ti.flags & kFirst) {
#pragma unroll
        for (int h = 0; h < NH; ++h) fac[h] = h < G ? ms.fac[st][h] : 0.f;
      }
      const float ksc = ms.ks[st][tid >> 4], vsc = ms.vs[st][tid >> 4];
      const bool seen = ksc >= 0.f && ti.tile * TT + tid < ti.len;
      const float lv = __log2f(vsc), iv = 1.f / vsc;
      float x[NH];
      bool raise = false;
#pragma unroll
      for (int cb = 0; cb < N; cb += 16) {
        float v[16];
        tmem_ld16(lane_base + buf * N + cb, v);
        tmem_wait_ld();
#pragma unroll
        for (int hl = 0; hl < 16 / STR; ++hl) {
          const int h = cb / STR + hl;
          float s = v[hl * STR + CC::QPARTS - 1];
#pragma unroll
          for (int i = CC::QPARTS - 2; i >= 0; --i) s = fmaf(s, 1.f / 16.f, v[hl * STR + i]);
          x[h] = seen ? fmaf(s, fac[h] * ksc, lv) : -INFINITY;
          raise |= h < G && x[h] - ref[h] > kLazy;     // the difference is exact where p could get too large
        }
      }
      // one thread decides for all whether an abort ends the work here
      if (tid == 0) ms.stop[buf] = *(volatile int*)&ms.abort;
      if (named_bar_or(1, kSoftThreads, raise)) {
        // a score far above the reference (always in a part's first tile): raise it to the tile's maximum
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          if (h >= G) break;
          float m = x[h];
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
          if (lane == 0) ms.red[w][h] = m;
        }
        named_bar_sync(1, kSoftThreads);
        float al[NH];
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          al[h] = 1.f;
          if (h >= G) continue;
          const float m = fmaxf(fmaxf(ms.red[0][h], ms.red[1][h]), fmaxf(ms.red[2][h], ms.red[3][h]));
          if (m > ref[h]) {
            al[h] = fast_exp2(ref[h] - m);
            ref[h] = m;
            l[h] *= al[h];
            if (STR == 8) {
              acc[h] *= al[h];
              lacc[h] *= al[h];
            }
          }
        }
        if (begun) {
          wait(&ms.pv_done[(t - 1) & 1], ((t - 1) >> 1) & 1);
          tc_fence_after();
#pragma unroll
          for (int cb = 0; cb < N; cb += 16) {
            float v[16];
            tmem_ld16(lane_base + 2 * N + cb, v);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] *= al[(cb + i) / STR];
            tmem_st16(lane_base + 2 * N + cb, v);
          }
          tmem_wait_st();
        }
        named_bar_sync(1, kSoftThreads);      // ms.red is free again
      }
      if (ms.stop[buf]) break;
      begun = true;
      if (t >= 2) wait(&ms.pv_done[buf], ((t - 2) >> 1) & 1);
      uint8_t* pb = dyn + off_p + buf * N * TT + pcol;
#pragma unroll
      for (int h = 0; h < NH; h += 2) {
        if (h >= G) break;
        const float a0 = fast_exp2(x[h] - (ref[h] == -INFINITY ? 0.f : ref[h]) + kPScale);
        const float a1 = h + 1 < G ? fast_exp2(x[h + 1] - (ref[h + 1] == -INFINITY ? 0.f : ref[h + 1]) + kPScale) : 0.f;
        l[h] = fmaf(a0, iv, l[h]);
        l[h + 1] = fmaf(a1, iv, l[h + 1]);
        // Two heads as a pair of f16 numbers: the upper byte of one is the e5m2 number that its lower bits are cut off
        // from, and what is left times 8 is exact.  bf16 outputs: what the first part leaves is taken from the f32 p, so
        // that f16 rounds an eighth of it, and the others are rounded: off by 2^-12 of p at most, 2^-16 as a rule (an f16
        // p: 2^-11 and 2^-13).  f32 outputs: all four parts of the f16 p, then of what its rounding left, 2^12 times (at
        // most half a step of 2^4).
        __half2 p2 = __floats2half2_rn(a0, a1), rest;
        if (STR == 8) {
          const float2 f = __half22float2(p2);
          rest = __floats2half2_rn((a0 - f.x) * 4096.f, (a1 - f.y) * 4096.f);
        }
#pragma unroll
        for (int i = 0; i < CC::PPARTS; ++i) {
          if (i == 4) p2 = rest;
          uint32_t bits = *reinterpret_cast<const uint32_t*>(&p2);
          if (STR == 4 && i > 0) bits += 0x00800080u;          // to the nearest, away from 0 on a tie
          const int n0 = h * STR + i, n1 = n0 + STR;
          pb[n0 * TT + ((pchunk ^ (n0 & 7)) << 4)] = (uint8_t)(bits >> 8);
          pb[n1 * TT + ((pchunk ^ (n1 & 7)) << 4)] = (uint8_t)(bits >> 24);
          const uint32_t top = bits & 0xff00ff00u;
          const __half2 cut = *reinterpret_cast<const __half2*>(&top);
          if (STR == 4 && i == 0) {
            const float2 f = __half22float2(cut);
            const float2 r = eight_times(make_float2(a0, a1), f);
            p2 = __floats2half2_rn(r.x, r.y);
          } else if ((i & 3) < 3) {
            p2 = __hmul2(__hsub2(p2, cut), __float2half2_rn(8.f));
          }
        }
      }
      if (!seen) {
        // a row that is not the sequence's: zeros, since 0 times what is stored there may be NaN
        wait_or_abort(&ms.v_full[st], (t / kVStages) & 1, &ms.abort, p.ctrl);
        uint4* row = reinterpret_cast<uint4*>(dyn + st * kStageV + tid * D);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) row[i] = make_uint4(0, 0, 0, 0);
      }
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive(&ms.p_full[buf]);
      if (!(ti.flags & kLast)) continue;

      // ---- end of the unit, or of this piece's share of it
      const size_t row0 = (size_t)ti.b * p.Hq + (size_t)ti.g * G;
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        if (h >= G) break;
        if (STR == 8) l[h] += lacc[h];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], o);
        if (lane == 0) ms.red[w][h] = l[h];
      }
      named_bar_sync(1, kSoftThreads);
      wait(&ms.pv_done[buf], (t >> 1) & 1);
      tc_fence_after();
#pragma unroll
      for (int cb = 0; cb < N; cb += 16) {
        float v[16];
        tmem_ld16(lane_base + 2 * N + cb, v);
        tmem_wait_ld();
#pragma unroll
        for (int hl = 0; hl < 16 / STR; ++hl) {
          const int h = cb / STR + hl;
          if (h >= G) continue;
          float O = head_of(v, hl);
          if (STR == 8) O += acc[h];
          const float L = (ms.red[0][h] + ms.red[1][h]) + (ms.red[2][h] + ms.red[3][h]);
          if (ti.slot < 0) {
            store_out_elem(p, (row0 + h) * D + tid, normalised(O, L));
            if (p.lse_out && tid == 0) p.lse_out[row0 + h] = lse_of(ref[h], L, kPScale);
          } else {
            p.part_o[((size_t)ti.slot * G + h) * D + tid] = O;
            if (tid == 0) p.part_ml[(size_t)ti.slot * G + h] = make_float2(ref[h], L);
          }
        }
      }
      if (ti.slot < 0 && tid < G) {           // for the merge kernel: heads with a NaN that their query does not bring
        const float L = (ms.red[0][tid] + ms.red[1][tid]) + (ms.red[2][tid] + ms.red[3][tid]);
        if (L != L && p.qfac[(size_t)ti.u * kMaxG + tid] < INFINITY) p.again[atomicAdd(p.ctl + 2, 1)] = ti.u * kMaxG + tid;
      }
      tc_fence_before();
      named_bar_sync(1, kSoftThreads);        // ms.red is free again
      if (ti.flags & kEnd) break;
    }
  }
  __syncthreads();
  if (w == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"((uint32_t)CC::TMEM) : "memory");
}

// ============================================================================
// merge of the parts of units that several blocks shared
// ============================================================================

// Blocks share the (unit, query head) pairs of the list.  Bound by the latency of
// two dependent loads: which parts, and the parts (M, l and O together, eight at a
// time).  Up to eight parts are a warp's business, a float4 of O per lane (a block
// for each took 22.8 us for 296 units of 8 heads in two parts, this 2.5).  For
// more, each of eight warps runs over every eighth part; then the eight results
// are added in order.
constexpr int kMergeWarps = 8;
constexpr int kMergeFew = 8;
constexpr int kMaxPieces = 2048;
constexpr int kPiecesPerBlock = 2;         // a first piece and a later one
// At most that many units of kMaxG heads for each block of the merge, whether a warp or the block takes them.
constexpr int kMaxRedo = kPiecesPerBlock * kMaxG * 2;

// A NaN code in a dimension that a head left out makes its score on the tensor cores NaN (the query's factor there is
// 0, and the rows come with every dimension that a head of the group kept).  So a head with a NaN that its query does
// not bring is formed again here, by one warp over the dimensions it kept: a token a lane for the scores, four dims of
// the output a lane for the values.  A NaN in a kept dimension shows again and ends the work; the first of them is
// looked through ahead, since a row that a NaN was appended to is NaN as a whole.  Rare, and slow: one head of 131072
// tokens 47 ms, 0.3 ms where its rows are NaN as a whole.
__device__ __forceinline__ void form_again(const PagedView& c, const DecodeP& p, int G, int u, int hh, int cols, int stride, int parts) {
  const int lane = threadIdx.x & 31, b = u / c.Hkv, g = u % c.Hkv;
  const size_t row = (size_t)b * p.Hq + (size_t)g * G + hh;
  const float fac = p.qfac[(size_t)u * kMaxG + hh];
  const uint8_t* q = p.qpart + ((size_t)u * cols + hh * stride) * D + lane;
  float x[4];                                // dims lane + 32 y
  uint32_t kept[4];
#pragma unroll
  for (int y = 0; y < 4; ++y) {
    x[y] = 0.f;
    for (int i = parts - 1; i >= 0; --i) x[y] = fmaf(x[y], 1.f / 16.f, e4m3x2_to_f32x2(q[i * D + 32 * y]).x);
    kept[y] = __ballot_sync(0xffffffffu, q[32 * y] != 0);
  }
  const int n = seq_tokens(c, p, b), mask = (1 << c.page_log2) - 1;
  const int first = kept[0] ? __ffs(kept[0]) - 1 : kept[1] ? __ffs(kept[1]) + 31 : kept[2] ? __ffs(kept[2]) + 63 : __ffs(kept[3]) + 95;
  auto page_of = [&](int t) {
    const int pid = t < n ? __ldg(c.table + (size_t)b * c.max_pages + (t >> c.page_log2)) : -1;
    return pid < c.n_pages ? pid : -1;
  };
  bool nan = false;
#pragma unroll 4
  for (int t = 16 * lane; t < n; t += 32 * 16) {                 // sixteen codes, of one page
    const int pid = page_of(t);
    if (pid < 0) continue;
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(c.k + c.kblock(pid, g) + ((size_t)first << c.page_log2) + (t & mask)));
    const uint32_t words[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 16; ++i) nan |= t + i < n && ((words[i >> 2] >> (8 * (i & 3))) & 0x7fu) == 0x7fu;
  }
  nan = __any_sync(0xffffffffu, nan);
  float M = nan ? NAN : -INFINITY, l = nan ? NAN : 0.f;
  float4 acc = nan ? make_float4(NAN, NAN, NAN, NAN) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int t0 = nan ? n : 0; t0 < n; t0 += 32) {
    const int t = t0 + lane, pid = page_of(t);
    const bool seen = pid >= 0;
    const size_t si = seen ? (size_t)pid * c.Hkv + g : 0;
    const uint8_t* key = c.k + (seen ? c.kblock(pid, g) + (t & mask) : 0);
    float s = 0.f;
#pragma unroll
    for (int y = 0; y < 4; ++y) {
#pragma unroll 1
      for (int i0 = 0; i0 < 32; i0 += 16) {                      // sixteen loads in flight
        uint8_t code[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
          code[i] = seen && ((kept[y] >> (i0 + i)) & 1u) ? key[(size_t)(i0 + i + 32 * y) << c.page_log2] : (uint8_t)0;
#pragma unroll
        for (int i = 0; i < 16; ++i) s = fmaf(__shfl_sync(0xffffffffu, x[y], i0 + i), e4m3x2_to_f32x2(code[i]).x, s);
      }
    }
    s = seen ? s * (fac * c.ks[si]) : -INFINITY;
    if (__any_sync(0xffffffffu, s != s)) {
      M = l = NAN;
      acc = make_float4(NAN, NAN, NAN, NAN);
      break;
    }
    float top = s;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    top = fmaxf(top, M);
    const float ref = top == -INFINITY ? 0.f : top, al = fast_exp2(M - ref), e = fast_exp2(s - ref);
    M = top;
    l = fmaf(l, al, e);
    acc.x *= al; acc.y *= al; acc.z *= al; acc.w *= al;
    const float w = seen ? e * c.vs[si] : 0.f;
#pragma unroll 1
    for (int i0 = 0; i0 < 32; i0 += 8) {
      uint32_t v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int pi = __shfl_sync(0xffffffffu, pid, i0 + i);
        v[i] = pi >= 0 ? reinterpret_cast<const uint32_t*>(c.v + c.vblock(pi, g) + (size_t)((t0 + i0 + i) & mask) * D)[lane] : 0u;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float wi = __shfl_sync(0xffffffffu, w, i0 + i);
        const float2 v0 = e4m3x2_to_f32x2((uint16_t)v[i]), v1 = e4m3x2_to_f32x2((uint16_t)(v[i] >> 16));
        acc.x = fmaf(wi, v0.x, acc.x); acc.y = fmaf(wi, v0.y, acc.y);
        acc.z = fmaf(wi, v1.x, acc.z); acc.w = fmaf(wi, v1.y, acc.w);
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  const size_t at = row * D + 4 * lane;
  store_out_elem(p, at, normalised(acc.x, l));
  store_out_elem(p, at + 1, normalised(acc.y, l));
  store_out_elem(p, at + 2, normalised(acc.z, l));
  store_out_elem(p, at + 3, normalised(acc.w, l));
  if (p.lse_out && lane == 0) p.lse_out[row] = lse_of(M, l, 0.f);
}

__global__ void __launch_bounds__(kMergeWarps * 32) paged_merge_kernel(const __grid_constant__ PagedView c, const __grid_constant__ DecodeP p, int G, int cols, int stride, int parts) {
  __shared__ __align__(16) float sum[kMergeWarps][D];
  __shared__ float2 ml[kMergeWarps];
  __shared__ int redo[kMaxRedo], n_redo;   // heads to form again among this block's: unit * kMaxG + head
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  if (tid == 0) n_redo = 0;
  __syncthreads();
  pdl_wait();
  int4 sp = p.split[blockIdx.x / G];       // along with their number: the list has room for more than the blocks
  const int n_jobs = p.ctl[1] * G, n_again = p.ctl[2];
  // whether a sum of weights is NaN and the query is not
  auto odd = [&](float L, int u, int hh) { return L != L && p.qfac[(size_t)u * kMaxG + hh] < INFINITY; };
  // units cut in eight parts or fewer: a warp each
#pragma unroll 1
  for (int job = blockIdx.x * kMergeWarps + w; job < n_jobs; job += gridDim.x * kMergeWarps) {
    const int hh = job % G;
    const int4 s1 = p.split[job / G];
    const int n = s1.z - s1.y + 1;
    if (n > kMergeFew) continue;
    float2 m[kMergeFew];
    float4 v[kMergeFew];
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kMergeFew; ++i) {
      m[i] = make_float2(-INFINITY, 0.f);
      v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < n) {
        const size_t slot = (size_t)(2 * (s1.y + i) + (i == 0 ? s1.w : 0)) * G + hh;
        m[i] = p.part_ml[slot];
        v[i] = *reinterpret_cast<const float4*>(p.part_o + slot * D + 4 * lane);
      }
    }
#pragma unroll
    for (int i = 0; i < kMergeFew; ++i) top = fmaxf(top, m[i].x);
    const float ref = top == -INFINITY ? 0.f : top;
    float L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kMergeFew; ++i) {
      const float f = fast_exp2(m[i].x - ref);
      L = fmaf(m[i].y, f, L);
      acc.x = fmaf(v[i].x, f, acc.x); acc.y = fmaf(v[i].y, f, acc.y);
      acc.z = fmaf(v[i].z, f, acc.z); acc.w = fmaf(v[i].w, f, acc.w);
    }
    if (odd(L, s1.x, hh)) {
      if (lane == 0) redo[atomicAdd(&n_redo, 1)] = s1.x * kMaxG + hh;
      continue;
    }
    const size_t row = (size_t)(s1.x / c.Hkv) * p.Hq + (size_t)(s1.x % c.Hkv) * G + hh;
    const size_t at = row * D + 4 * lane;
    store_out_elem(p, at, normalised(acc.x, L));
    store_out_elem(p, at + 1, normalised(acc.y, L));
    store_out_elem(p, at + 2, normalised(acc.z, L));
    store_out_elem(p, at + 3, normalised(acc.w, L));
    if (p.lse_out && lane == 0) p.lse_out[row] = lse_of(top, L, kPScale);
  }
  // the others: a block each
#pragma unroll 1
  for (int job = blockIdx.x; job < n_jobs; job += gridDim.x) {
    const int hh = job % G;
    if (job != (int)blockIdx.x) sp = p.split[job / G];
    const int n = sp.z - sp.y + 1;
    if (n <= kMergeFew) continue;
    float M = -INFINITY, L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int i0 = w; i0 < n; i0 += 8 * kMergeWarps) {
      float2 m[8];
      float4 v[8];
#pragma unroll
      for (int z = 0; z < 8; ++z) {
        const int i = i0 + z * kMergeWarps;
        m[z] = make_float2(-INFINITY, 0.f);
        v[z] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i < n) {
          const size_t slot = (size_t)(2 * (sp.y + i) + (i == 0 ? sp.w : 0)) * G + hh;
          m[z] = p.part_ml[slot];
          v[z] = *reinterpret_cast<const float4*>(p.part_o + slot * D + 4 * lane);
        }
      }
      float top = M;
#pragma unroll
      for (int z = 0; z < 8; ++z) top = fmaxf(top, m[z].x);
      const float ref = top == -INFINITY ? 0.f : top, al = fast_exp2(M - ref);
      M = top;
      L *= al;
      acc.x *= al; acc.y *= al; acc.z *= al; acc.w *= al;
#pragma unroll
      for (int z = 0; z < 8; ++z) {
        const float f = fast_exp2(m[z].x - ref);
        L = fmaf(m[z].y, f, L);
        acc.x = fmaf(v[z].x, f, acc.x); acc.y = fmaf(v[z].y, f, acc.y);
        acc.z = fmaf(v[z].z, f, acc.z); acc.w = fmaf(v[z].w, f, acc.w);
      }
    }
    *reinterpret_cast<float4*>(&sum[w][4 * lane]) = acc;
    if (lane == 0) ml[w] = make_float2(M, L);
    __syncthreads();
    float all = 0.f;                         // NaN as the whole sum is
#pragma unroll
    for (int z = 0; z < kMergeWarps; ++z) all += ml[z].y;
    if (odd(all, sp.x, hh)) {
      if (tid == 0) redo[atomicAdd(&n_redo, 1)] = sp.x * kMaxG + hh;
    } else if (tid < D) {
      float top = -INFINITY;
#pragma unroll
      for (int z = 0; z < kMergeWarps; ++z) top = fmaxf(top, ml[z].x);
      const float ref = top == -INFINITY ? 0.f : top;
      float O = 0.f, Ls = 0.f;
#pragma unroll
      for (int z = 0; z < kMergeWarps; ++z) {
        const float f = fast_exp2(ml[z].x - ref);
        O = fmaf(sum[z][tid], f, O);
        Ls = fmaf(ml[z].y, f, Ls);
      }
      const size_t row = (size_t)(sp.x / c.Hkv) * p.Hq + (size_t)(sp.x % c.Hkv) * G + hh;
      store_out_elem(p, row * D + tid, normalised(O, Ls));
      if (p.lse_out && tid == 0) p.lse_out[row] = lse_of(top, Ls, kPScale);
    }
    __syncthreads();
  }
  // formed again at the end, in one place: calls among the merges cost every step 1 us
  __syncthreads();
  const int mine = n_redo, n_jobs_again = mine + max(0, (n_again - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x);
#pragma unroll 1
  for (int i = w; i < n_jobs_again; i += kMergeWarps) {
    const int what = i < mine ? redo[i] : p.again[blockIdx.x + (i - mine) * gridDim.x];
    form_again(c, p, G, what / kMaxG, what % kMaxG, cols, stride, parts);
  }
}

// ---------------------------------------------------------------- host side
struct Layout {
  size_t umask, qpart, qfac, prefix, ctl, part_ml, part_o, split, again, total;
};

// The workspace does not depend on the output type: room for the widest operands.
Layout layout_of(int B, int Hkv, int G, int blocks) {
  const int n_units = B * Hkv, pieces = kPiecesPerBlock * blocks;
  const int cols = G > 4 ? 64 : 32;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t r = at;
    at = (at + bytes + 255) & ~(size_t)255;
    return r;
  };
  Layout y;
  y.umask = take((size_t)n_units * sizeof(uint4));
  y.qpart = take((size_t)n_units * cols * D);
  y.qfac = take((size_t)n_units * kMaxG * 4);
  y.prefix = take((size_t)(B + 1) * 4);
  y.ctl = take(3 * 4);
  y.part_ml = take((size_t)2 * pieces * G * sizeof(float2));
  y.part_o = take((size_t)2 * pieces * G * D * 4);
  y.split = take((size_t)pieces * sizeof(int4));
  y.again = take((size_t)n_units * kMaxG * 4);
  y.total = at;
  return y;
}

int attend_blocks(int per_sm) {
  const int n = per_sm * device_sm_count();
  return n < kMaxPieces / kPiecesPerBlock ? n : kMaxPieces / kPiecesPerBlock;
}

template <typename T>
int launch_select(const PagedView& c, const DecodeP& p, int G, int NH, int stride, int parts, cudaStream_t st) {
  // As many sequences a block as leave one or two blocks an SM: P is read once for all of them, and where there is
  // one, an attention block fits beside it and fetches its first tiles.
  // With two sequences a block or more the selection itself is what takes long, and two blocks an SM overlap
  // (1560 units of 8 heads: 78 us in one block an SM, 57 in two; a step of 256 units of 4 heads: 41.2 and 39.0).
  const int sms = device_sm_count();
  const int waves = (long long)c.B * c.Hkv > sms ? 2 : 1;
  const int each = waves * sms / c.Hkv > 0 ? waves * sms / c.Hkv : 1;                 // blocks a head
  const int group = (c.B + each - 1) / each;
  const dim3 grid((c.B + group - 1) / group, c.Hkv);
  const auto kernel = paged_select_kernel<T>;
  const int rc = set_largest_carveout(reinterpret_cast<const void*>(kernel), "paged_select_kernel");
  if (rc != AQUA_OK) return rc;
  const cudaError_t e = launch_pdl(kernel, grid, dim3(kSelThreads), 0, st, c, p, G, NH, stride, parts, group);
  if (e != cudaSuccess) return set_error(AQUA_ERR_CUDA, "paged_select_kernel: %s", cudaGetErrorString(e));
  return check_launch("paged_select_kernel");
}

template <int STR, int NH>
int launch_step(const PagedView& c, const DecodeP& p, int G, bool bf16, cudaStream_t st) {
  using CC = Cols<STR, NH>;
  const int smem = CC::smem(c.m), blocks = attend_blocks(CC::CTAS);
  int rc = set_smem_limit(paged_attend_kernel<STR, NH>, smem, "paged_attend_kernel");
  if (rc != AQUA_OK) return rc;
  // value pages as rows of 128 bytes (64 columns of two), a page a box
  CUtensorMap vmap;
  rc = encode_tmap_bf16_2d(&vmap, c.v, D / 2, (uint64_t)c.n_pages * c.Hkv << c.page_log2, D, D / 2, c.page, true);
  if (rc != AQUA_OK) return rc;
  rc = bf16 ? launch_select<__nv_bfloat16>(c, p, G, NH, STR, CC::QPARTS, st) : launch_select<float>(c, p, G, NH, STR, CC::QPARTS, st);
  if (rc != AQUA_OK) return rc;
  cudaError_t e = launch_pdl(paged_attend_kernel<STR, NH>, dim3(blocks), dim3(kThreads), smem, st, vmap, c, p, G);
  if (e != cudaSuccess) return set_error(AQUA_ERR_CUDA, "paged_attend_kernel: %s", cudaGetErrorString(e));
  if ((rc = check_launch("paged_attend_kernel")) != AQUA_OK) return rc;
  rc = set_largest_carveout(reinterpret_cast<const void*>(paged_merge_kernel), "paged_merge_kernel");
  if (rc != AQUA_OK) return rc;
  e = launch_pdl(paged_merge_kernel, dim3(blocks), dim3(kMergeWarps * 32), 0, st, c, p, G, CC::N, STR, CC::QPARTS);
  if (e != cudaSuccess) return set_error(AQUA_ERR_CUDA, "paged_merge_kernel: %s", cudaGetErrorString(e));
  return check_launch("paged_merge_kernel");
}

}  // namespace

size_t paged_decode_workspace_bytes(int B, int Hkv, int G) { return layout_of(B, Hkv, G, attend_blocks(2)).total; }

int launch_paged_decode(const PagedView& c, const int32_t* len, const void* q, bool bf16, const Strides& qs,
                        const float* P, const RopeView& rope, int Hq, int k, float scale, void* out, bool out_bf16,
                        int32_t* sel_out, float* qproj_out, float* lse_out, void* ws, cudaStream_t st) {
  const int G = Hq / c.Hkv;
  const Layout y = layout_of(c.B, c.Hkv, G, attend_blocks(2));
  uint8_t* base = static_cast<uint8_t*>(ws);
  DecodeP p;
  p.len = len; p.q = q; p.qs = qs; p.P = P; p.rope = rope; p.Hq = Hq; p.k = k; p.scale = scale;
  p.out = out; p.out_bf16 = out_bf16; p.sel_out = sel_out; p.qproj_out = qproj_out; p.lse_out = lse_out;
  p.ctrl = c.ctrl;
  p.umask = reinterpret_cast<uint4*>(base + y.umask);
  p.prefix = reinterpret_cast<int32_t*>(base + y.prefix);
  p.ctl = reinterpret_cast<int32_t*>(base + y.ctl);
  p.qpart = base + y.qpart;
  p.qfac = reinterpret_cast<float*>(base + y.qfac);
  p.part_ml = reinterpret_cast<float2*>(base + y.part_ml);
  p.part_o = reinterpret_cast<float*>(base + y.part_o);
  p.split = reinterpret_cast<int4*>(base + y.split);
  p.again = reinterpret_cast<int32_t*>(base + y.again);
  if (out_bf16) return G > 4 ? launch_step<4, 8>(c, p, G, bf16, st) : launch_step<4, 4>(c, p, G, bf16, st);
  return G > 4 ? launch_step<8, 8>(c, p, G, bf16, st) : launch_step<8, 4>(c, p, G, bf16, st);
}

}  // namespace aqua
