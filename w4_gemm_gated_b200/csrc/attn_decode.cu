// Attention of one new token per sequence over the paged cache.
//
//   out_h = sum_t p_t v_t,  p = softmax(scale q_h . k_t)
//
// Each cached byte is read once for every 8 or 16 of the query heads that share it
// (two operations per value and head), so HBM bounds it in principle, and does for
// bf16 and groups of up to 8: 2 sequences of up to 131,072 tokens, 8 heads of 128,
// 800 MB in 128 us, 6.2 TB/s.  Quantised caches take a few instructions per code,
// which bound them where no heads share them (int4, 32 x 4099, 32 heads: 272 MB in 66
// us, 4.1 TB/s, at 58 % of the issue rate).  Short batches are bound by the chain from
// the lengths over the page table to the data and by the joins (int8, 16 x 2048: 36
// MB in 17 us).
//
// Work.  A unit is one (sequence, kv head) with up to 8 NT query heads; its
// tokens are cut into tiles of TILE.  All units' tiles in order form one line
// (with a step for each unit besides), which is cut into equal runs, one per CTA
// and in it one per warp, by the lengths alone (every CTA sums them up): ragged
// batches load the machine evenly, a long sequence is spread over many warps, and
// a warp takes many short ones without meeting anybody.  Where every unit is short
// the CTAs' borders move to units' borders.  A warp streams its run through its own
// ring of shared-memory stages (16-byte asynchronous copies, rows past a sequence's
// end filled with zeros), so that copies cross the units' borders and never wait
// for another warp.
//
// Arithmetic.  Tensor-core products over 16 tokens with the query heads as the 8
// columns: S = K q (rows: tokens), then O^T += V^T P with P's layout turned by
// movmatrix.  Running reference, sum and output of a softmax in fp32, in powers of
// two; they are rescaled only when a weight passes the reference by 2^kSlack.
// The operands of the second product are the weights times their values' scales
// as two bf16 parts each (relative 2^-17, 2^-9 of the output's own rounding).  One
// fp16 part costs less (int4, 32 x 4099, 32 heads: 63 us) but has 2^-11, and too short a
// range: a token of large weight whose values are small or nothing, as padding's are,
// brings the others, which the output then consists of, among its subnormals.
// The sum in the denominator is of the unrounded weights.  Codes with an offset, u
// = c + 128 or c + 8, are subnormals as they are: 2^-24 u (2^-24 16 u) of fp16,
// beside q, 2^-133 u of bf16, beside the weights.  What they are too large by the
// scores' sums start from, negative; for the output one product-sum brings the
// operand to 2^-6 c, exactly.
//
// Joining.  A warp whose run starts or ends inside a unit leaves (maximum, sum,
// output) in shared memory; the CTA joins the pieces of a unit in order, and
// a unit that crosses CTAs is joined, again in order, by whichever of them
// arrives last (a counter per unit, left at zero): no launch waits, and the
// result does not depend on who is last.
#include <atomic>

#include "kv_cache.cuh"

namespace spear {

struct AttnArgs {
  KvView c;
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  float* lse;
  const int* table;
  const int* lens;
  long long ld_q, ld_out;
  int ld_table, max_len, n_seqs, heads, group;
  int blocks;   // units per kv head: ceil(group / (8 NT))
  float scale;  // times log2(e)
  WsHeader* hdr;
  int ctas;      // at most
  int* tickets;  // one per CTA: arrivals at the unit that crosses out of it first; two per CTA: at its parts' groups
  float* parts;  // two pieces per CTA
};

constexpr int kRadix = 16;    // parts of a unit joined at once; more are joined in groups of as many first
constexpr int kMinTiles = 2;  // tiles a warp should have before more CTAs take part
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.f;  // how far, in powers of two, a weight may lie above 1
constexpr int kShort = 32;    // tiles up to which a unit stays in one CTA

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Wait until at most N of this thread's copy groups are in flight.
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int N>
__device__ __forceinline__ void lds(uint32_t addr, uint32_t (&w)[N]) {
  if constexpr (N == 1) asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(addr) : "memory");
  if constexpr (N == 2) asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr) : "memory");
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ float lds_half(uint32_t addr) {
  unsigned short v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
  return __half2float(__ushort_as_half(v));
}
__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ float exp2_(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// D(16x8, fp32) += A(16x16) . B(16x8), both fp16 (F16) or both bf16.
template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else mma_bf16_16816(d, a, b0, b1);
}
// Codes as 16-bit floats: an integer u < 256 in the low bits is 2^-24 u of fp16 and
// 2^-133 u of bf16, exactly.  int8 codes, offset to u = c + 128 by kFlip, two bytes of
// a word at a time; int4 codes u = c + 8 from bits 0-3 as u and from bits 4-7, without a
// shift, as 16 u.
constexpr uint32_t kFlip = 0x80808080u;
constexpr float kUnit = 16777216.f;  // 2^24
template <int SEL>
__device__ __forceinline__ uint32_t two_bytes(uint32_t w) {
  return __byte_perm(w, 0u, SEL);  // 5 and 7 pick 0
}
__device__ __forceinline__ uint32_t low4(uint32_t w) { return w & 0x000F000Fu; }
__device__ __forceinline__ uint32_t high4(uint32_t w) { return w & 0x00F000F0u; }
// The offsets 8 and 128 (of 16 u too), negative, as fp16 operands.
constexpr uint32_t kLess8 = 0x80088008u, kLess128 = 0x80808080u;
// bf16 pairs: a b + c.
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
// Codes 2^-133 u of bf16, times 2^127, less the offset's 2^-6 8 or 2^-6 128.
constexpr uint32_t kOff8 = 0xBE00BE00u, kOff128 = 0xC000C000u;
constexpr float kValue = 64.f;  // 2^6
__device__ __forceinline__ uint32_t centred(uint32_t u, uint32_t off) { return fma_bf16x2(u, 0x7F007F00u, off); }
// Whether one of the 16 bf16 values of these words is infinite or NaN: 0 times it is NaN.
__device__ __forceinline__ bool any_beyond(const uint32_t (&v)[4][4]) {
  uint32_t t[2] = {0u, 0u};
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int w = 0; w < 4; ++w) t[w & 1] = fma_bf16x2(v[k][w], 0u, t[w & 1]);
  return t[0] | t[1];
}
// Two bf16 values, infinities and NaN as 0.
__device__ __forceinline__ uint32_t finite_part(uint32_t w) {
  return w & ~__vcmpeq2(w & 0x7F807F80u, 0x7F807F80u);
}
// Two values as bf16 pairs: rounded, and what that leaves.
__device__ __forceinline__ void split_bf16(float a, float b, uint32_t& high, uint32_t& low) {
  high = pack_bf16x2(a, b);
  low = pack_bf16x2(a - __uint_as_float(high << 16), b - __uint_as_float(high & 0xFFFF0000u));
}

// Layout of a unit's tiles in shared memory and in the fragments.
template <int KIND, int DIM>
struct Lay {
  static constexpr int RB = DIM * kv_bits(KIND) / 8;       // bytes of a row
  static constexpr int TS = RB >= 128 ? 1 : 2;             // blocks of 16 tokens per tile
  static constexpr int TILE = 16 * TS;
  static constexpr bool QUANT = KIND != SPEAR_KV_BF16;
  static constexpr int SIDE = TILE * RB;                   // K (or V) bytes of a stage
  static constexpr int STAGE = 2 * SIDE + (QUANT ? 4 * TILE : 0);
  // dims of a lane's run in O: dim = (a / (VL / 2)) 8 VL + rho VL + 2 (a % (VL / 2)) + {0, 1}
  static constexpr int VL = KIND == SPEAR_KV_BF16 ? 8 : KIND == SPEAR_KV_INT8 ? (DIM >= 128 ? 16 : 8) : DIM / 8;
  static constexpr int VW = VL * kv_bits(KIND) / 32;       // 32-bit words of such a run
  static constexpr int KW = DIM * kv_bits(KIND) / 128 >= 4 ? 4 : DIM * kv_bits(KIND) / 128;  // words per K load
  static constexpr int KI = DIM * kv_bits(KIND) / 128 / KW;                                 // K loads per row

  // Row r of a fragment's 16 is token tok(r) of the block, and the 16-byte
  // chunks of a row are permuted by xk / xv, so that the 8 rows x 4 lanes of a
  // K load and the 4 tokens x 8 lanes of a V load each meet all banks.
  static __device__ __forceinline__ int tok(int r) {
    if constexpr (RB >= 128) return r;
    const int c = (r >> 1) & 3;
    return (r & 8) + ((r & 1) ? 4 + (RB == 64 ? c ^ 1 : (c + 2) & 3) : c);
  }
  static __device__ __forceinline__ int xk(int t) { return RB >= 128 ? (t & 1) << 2 : RB == 64 ? t & 2 : 0; }
  static __device__ __forceinline__ int xv(int t) { return RB >= 128 ? ((t >> 1) & 3) << 1 : RB == 64 ? t & 2 : 0; }
};

__device__ __forceinline__ int clamp_len(const AttnArgs& p, int b) {
  const int n = p.lens[b];
  return n < 0 ? 0 : min(n, p.max_len);
}

// A place on the line: sequence, kv head, block of its query heads, tile of the unit.
struct Place {
  int b, head, blk, j, nt, len;
};

template <int TILE>
__device__ __forceinline__ void advance(const AttnArgs& p, Place& c) {
  if (++c.j < c.nt) return;
  c.j = 0;
  if (++c.blk < p.blocks) return;
  c.blk = 0;
  if (++c.head < p.c.heads) return;
  c.head = 0;
  do {
    if (++c.b >= p.n_seqs) return;
    c.len = clamp_len(p, c.b);
    c.nt = (c.len + TILE - 1) / TILE;
  } while (c.nt == 0);
}

// A warp's unfinished part of a unit.
struct Piece {
  unsigned start;  // the unit's begin on the line, which names the unit
  int nt;          // its tiles
  int from, to;    // tiles [from, to); to = 0: no piece
  int b, h0, num;  // its sequence, its first query head and their number
};

// Parts of a unit to be joined: n of them from CTA `first`, `every` apart.
struct Job {
  int c0;  // the unit's first CTA
  int first, every, n;
  bool mine, group;  // this CTA joins them; they are a group, more is to come
};

// A line of `total` cut into `parts` runs of q or q + 1.
struct Cut {
  unsigned q, more;  // the first `more` runs are one longer
  __device__ __forceinline__ Cut(unsigned total, unsigned parts) : q(total / parts), more(total - q * parts) {}
  __device__ __forceinline__ unsigned begin(unsigned w) const { return q * w + min(w, more); }
  __device__ __forceinline__ int owner(unsigned t) const {  // q > 0
    const unsigned border = (q + 1) * more;
    return t < border ? t / (q + 1) : more + (t - border) / q;
  }
};

// Warps of a CTA and CTAs of an SM.  Two CTAs, so that one streams while the other
// starts or joins (bf16, 64 x 4096: one of 8 warps 108 us, two of 4 101, four of 2
// 103).  Quantised kinds are bound by their arithmetic and take 16 warps where 128
// registers do (two of 8; with two of 4 int8 of 16 x 2048 takes 17.2 us, not 16.1, and
// int4 of 32 x 4099 with 32 heads 11 % more).
constexpr bool attn_small(int kind, int dim, int nt) { return kind != SPEAR_KV_BF16 && dim < 256 && nt == 1; }
constexpr int attn_warps(int kind, int dim, int nt) { return attn_small(kind, dim, nt) ? 8 : 4; }
constexpr int attn_per_sm(int kind, int dim) {  // at most 2, which the workspace counts on
  return kind == SPEAR_KV_BF16 && dim == 256 ? 1 : 2;
}

// Shared memory of a CTA: per warp a ring of stages and the place of a first
// piece.  227 KB per SM less 1 KB that each CTA takes besides, and 1 KB for the
// kernel's static arrays.
template <int KIND, int DIM, int NT>
struct Room {
  using L = Lay<KIND, DIM>;
  static constexpr int W = attn_warps(KIND, DIM, NT), PER_SM = attn_per_sm(KIND, DIM);
  static constexpr int PIECE = (8 * NT * (DIM + 2) + 3) / 4 * 4;  // floats: output, maximum, sum of each head
  static constexpr int ROOM = (227 * 1024 / PER_SM - 2048) / W - PIECE * 4;
  static constexpr int STAGES = ROOM / L::STAGE < 6 ? ROOM / L::STAGE : 6;
  static constexpr int RING = STAGES * L::STAGE;
  static constexpr int BYTES = W * (RING + PIECE * 4);
  static_assert(STAGES >= 2 && RING >= PIECE * 4, "a last piece takes the ring's place");
};

constexpr int kMaxSeqs = 4096;

// EH: columns of each lane's pair that can be heads; 1: only even columns are, and odd
// ones take the weights' low parts.
template <int KIND, int DIM, int NT, int EH, int W, int PER_SM>
__global__ void __launch_bounds__(W * 32, PER_SM) attn_kernel(const __grid_constant__ AttnArgs p) {
  using L = Lay<KIND, DIM>;
  using R = Room<KIND, DIM, NT>;
  static_assert(R::BYTES >= 8 * (kMaxSeqs + 1), "the line lies in the rings' place");
  constexpr int TILE = L::TILE, TS = L::TS, RB = L::RB, MT = DIM / 16;
  constexpr unsigned ALL = 0xFFFFFFFFu;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ unsigned scan_sum[W], scan_live[W];
  __shared__ int scan_max[W];
  __shared__ Piece pieces[2 * W];  // a warp's first (unit begun before it), its last
  __shared__ Job jobs[2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, rho = lane >> 2, cl = lane & 3;
  const int units = p.c.heads * p.blocks;
  after_previous();

  // ---- the line -----------------------------------------------------------------------
  // Every unit takes as many steps of it as it has tiles and one before them, since
  // to begin and to end a unit costs about what a tile does (a warp that got the 28
  // units of a one-token sequence for its 28 tiles took half as long again).
  // Up to 32 sequences: one per lane, in every warp alike.  More: in shared
  // memory, in the rings' place, a run of `per` to each thread.
  const bool few = p.n_seqs <= 32;
  unsigned* before = reinterpret_cast<unsigned*>(smem);  // steps of one unit of each sequence before it, n_seqs + 1
  unsigned* seqs = before + p.n_seqs + 1;                // sequences before it that have tokens
  int len_l = 0, nt_l = 0;                               // few: this lane's sequence
  unsigned before_l = 0, total, all_live = 0;
  int longest = 0;                                       // tiles of the longest unit
  {
    const int per = few ? 1 : (p.n_seqs + W * 32 - 1) / (W * 32);
    const int b0 = few ? lane : tid * per, b1 = min(b0 + per, p.n_seqs);
    unsigned sum = 0, live = 0;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      const int n = p.lens[b];
      if (blockIdx.x == 0 && (n < 0 || n > p.max_len)) report_status(p.hdr, SPEAR_ERR_DEVICE_CHECK);
      len_l = min(max(n, 0), p.max_len);
      nt_l = (len_l + TILE - 1) / TILE;
      if (!few) before[b] = nt_l;
      sum += nt_l + (nt_l > 0);
      live += nt_l > 0;
      longest = max(longest, nt_l);
    }
    auto scan = [&](unsigned v) {  // of the lanes before this one and this one
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const unsigned o = __shfl_up_sync(ALL, v, d);
        if (lane >= d) v += o;
      }
      return v;
    };
    const unsigned inc = scan(sum);
    longest = __reduce_max_sync(ALL, longest);
    before_l = inc - sum;
    total = __shfl_sync(ALL, inc, 31);
    if (lane < 2) pieces[2 * warp + lane].to = 0;
    if (!few) {
      const unsigned inc_live = scan(live);
      if (lane == 31) scan_sum[warp] = inc, scan_live[warp] = inc_live, scan_max[warp] = longest;
      __syncthreads();
      unsigned off = before_l, off_live = inc_live - live;
      total = 0;
#pragma unroll 1
      for (int w = 0; w < W; ++w) {
        if (w < warp) off += scan_sum[w], off_live += scan_live[w];
        total += scan_sum[w];
        all_live += scan_live[w];
        longest = max(longest, scan_max[w]);
      }
#pragma unroll 1
      for (int b = b0; b < b1; ++b) {
        const unsigned nt = before[b];
        before[b] = off;
        seqs[b] = off_live;
        off += nt + (nt > 0);
        off_live += nt > 0;
      }
      if (tid == 0) before[p.n_seqs] = total;
      __syncthreads();
    }
  }
  const unsigned seq_units = units * (few ? __popc(__ballot_sync(ALL, nt_l > 0)) : all_live);
  total *= units;
  // sequences without tokens
#pragma unroll 1
  for (int b = blockIdx.x; b < p.n_seqs; b += gridDim.x)
    if (few ? __shfl_sync(ALL, nt_l, b) == 0 : before[b] == before[b + 1]) {
#pragma unroll 1
      for (int i = tid; i < p.heads * DIM / 8; i += W * 32)
        *reinterpret_cast<uint4*>(p.out + b * p.ld_out + 8 * i) = make_uint4(0u, 0u, 0u, 0u);
      if (p.lse)
#pragma unroll 1
        for (int h = tid; h < p.heads; h += W * 32) p.lse[(long long)b * p.heads + h] = -INFINITY;
    }
  // ---- this CTA's and this warp's run ------------------------------------------------
  // Where no unit is longer than kShort tiles, CTAs take whole units: the borders
  // of even runs move on to the next unit's start.  A CTA may then have up to
  // kShort tiles more than its share, which costs no more than joining a unit
  // across CTAs does and saves that (7 sequences to 1001 tokens, 2 heads of 64: 9.9 us,
  // 11.2 with joins; a single sequence of 97, 8 heads, pays for it: 6.6 us, 6.2).
  const bool aligned = longest <= kShort;
  const unsigned ctas = min(gridDim.x, aligned ? min(total, (unsigned)(p.n_seqs * units))
                                               : (total + kMinTiles * W - 1) / (kMinTiles * W));
  if (blockIdx.x >= ctas) return;  // nothing for this CTA
  // Step t < total: the tile that comes at it or next; r: steps into its unit;
  // starts: units that start before t.
  auto place = [&](unsigned t, unsigned& r, unsigned& starts) {
    Place c;
    unsigned first;  // the sequence's first step
    if (few) {
      const unsigned live = __ballot_sync(ALL, nt_l > 0);
      c.b = 31 - __clz(__ballot_sync(ALL, nt_l > 0 && before_l * units <= t));
      first = __shfl_sync(ALL, before_l, c.b) * units;
      c.nt = __shfl_sync(ALL, nt_l, c.b);
      c.len = __shfl_sync(ALL, len_l, c.b);
      starts = __popc(live & ((1u << c.b) - 1u)) * units;
    } else {
      // the last b with before[b] * units <= t, 32 candidates at a time
      int b = 0;
#pragma unroll 1
      for (int step = p.n_seqs > 1024 ? 1024 : 32; step > 0; step >>= 5) {
        const int i = b + lane * step;
        b += step * (31 - __clz(__ballot_sync(ALL, i < p.n_seqs && before[i] * units <= t)));
      }
      c.b = b;
      first = before[b] * units;
      c.nt = before[b + 1] - before[b] - 1;
      c.len = clamp_len(p, b);
      starts = seqs[b] * units;
    }
    const unsigned u = (t - first) / (c.nt + 1);
    r = t - first - u * (c.nt + 1);
    starts += u + (r > 0);
    c.j = r ? r - 1 : 0;
    c.head = u;
    c.blk = 0;
    if (p.blocks > 1) {
      c.head = u / p.blocks;
      c.blk = u - c.head * p.blocks;
    }
    return c;
  };
  const Cut cut(total, ctas);
  unsigned c_begin = cut.begin(blockIdx.x), c_end = cut.begin(blockIdx.x + 1);
  unsigned start = 0;  // the begin of the unit that is worked on
  int n = 0;           // tiles
  Place in = {};       // next tile to copy
#pragma unroll 1
  for (int k = aligned ? 0 : 2; k < 4; ++k) {  // the CTA's begin and end, this warp's begin, and its end
    const Cut mine(c_end - c_begin, W);
    const unsigned t = k == 0 ? c_begin : k == 1 ? c_end : c_begin + mine.begin(k == 2 ? warp : warp + 1);
    unsigned r = 0, starts = seq_units;
    Place c = {};
    if (t < total) c = place(t, r, starts);
    const unsigned up = r ? t + c.nt + 1 - r : t;  // the next unit's start
    if (k == 0) {
      c_begin = up;
    } else if (k == 1) {
      c_end = up;
    } else if (k == 2) {
      in = c;
      start = t - r;
      n = c_begin + mine.begin(warp + 1) - t;  // steps
      if (t + n <= start + c.nt + 1) {         // in one unit
        n -= r == 0 && n > 0;
        break;
      }
      n = starts - t;  // tiles before the run, to be taken from those before its end
    } else {
      n += t - starts;
    }
  }
  Place at = in;  // tile to work on
  if (!few) __syncthreads();  // the rings take over `before`'s place

  uint8_t* ring = smem + (size_t)warp * (R::RING + R::PIECE * 4);
  float* first_piece = reinterpret_cast<float*>(ring + R::RING);
  float* last_piece = reinterpret_cast<float*>(ring);  // once the run is through
  const uint32_t ring_a = smem_u32(ring);

  // 32 entries of a sequence's row of the page table, one per lane
  int pg = 0, pg_seq = -1, pg_first = 0;
  auto page_of = [&](const Place& c, int t) {
    const int i = t >> p.c.log_page;
    if (c.b != pg_seq || (unsigned)(i - pg_first) >= 32u) {
      pg_seq = c.b;
      pg_first = i;
      pg = i + lane <= (c.len - 1) >> p.c.log_page ? p.table[(long long)c.b * p.ld_table + i + lane] : 0;
    }
    return __shfl_sync(0xFFFFFFFFu, pg, i - pg_first);
  };
  // A lane's chunk of a block's first 512 bytes; the next 512 bytes lie STEP rows on.
  constexpr int CPR = RB / 16, STEP = 32 / CPR;
  const int c_row = lane / CPR, c_ch = lane % CPR;
  const uint32_t k_dst = c_row * RB + ((c_ch ^ L::xk(c_row)) << 4);
  const uint32_t v_dst = c_row * RB + ((c_ch ^ L::xv(c_row)) << 4) + L::SIDE;
  const uint8_t* k_src = p.c.k + lane * 16;
  const uint8_t* v_src = p.c.v + lane * 16;
  // even lanes: 8 scales each of K, odd ones: of V
  const __half* s_src = L::QUANT ? (lane & 1 ? p.c.vs : p.c.ks) + (lane >> 1) * 8 : nullptr;
  const uint32_t s_dst = 2 * L::SIDE + (lane & 1) * 2 * TILE + (lane >> 1) * 16;
  // NB blocks of 16 tokens that lie in one page, from block s of the tile on;
  // rows past the first `rows` of the last one (`part`), and pages that are none, are zeros.
  auto copy_blocks = [&](uint32_t stage, int s, int t, int rows, auto nb, auto part) {
    constexpr int NB = decltype(nb)::value;
    const int entry = page_of(in, t);
    const bool ok = (unsigned)entry < (unsigned)p.c.n_pages;
    if (!ok && lane == 0) report_status(p.hdr, SPEAR_ERR_DEVICE_CHECK);
    const uint32_t page = ok ? entry : 0;
    const int row = (in.head << p.c.log_page) + (t & (p.c.page_size - 1));  // in the page
    const long long at_row = page_at(page, p.c.page_step) * 16 + row * RB;
    const uint8_t *ks = k_src + at_row, *vs = v_src + at_row;
    const uint32_t d = stage + 16 * s * RB;
    const int live = ok ? rows - c_row : 0, all = ok ? 16 : 0;
#pragma unroll
    for (int i = 0; i < NB * RB / 32; ++i) {
      const int bytes = decltype(part)::value ? (i * STEP < live ? 16 : 0) : all;
      cp_async16(d + (k_dst ^ (L::xk(i * STEP) << 4)) + i * 512, ks + i * 512, bytes);
      cp_async16(d + (v_dst ^ (L::xv(i * STEP) << 4)) + i * 512, vs + i * 512, bytes);
    }
    if constexpr (L::QUANT) {
      if (lane < 4 * NB)  // 8 scales each, of K and of V in turn
        cp_async16(stage + s_dst + 32 * s, s_src + page_at(page, p.c.scale_step) * 8 + row, all);
    }
  };
  auto copy_tile = [&](uint32_t stage) {
    const int t = in.j * TILE, rows = in.len - t;
    if (rows >= TILE && (TS == 1 || p.c.log_page > 4)) {
      copy_blocks(stage, 0, t, 0, std::integral_constant<int, TS>{}, std::false_type{});
    } else {
#pragma unroll 1
      for (int s = 0; s < TS && 16 * s < rows; ++s)
        copy_blocks(stage, s, t + 16 * s, rows - 16 * s, std::integral_constant<int, 1>{}, std::true_type{});
    }
  };

  // ---- the run ------------------------------------------------------------------------
  float acc[MT][NT][4], m[NT][2], l[NT][2];
  float kfix[NT][2];        // quantised: what the scores' sums start from
  float q_scale[NT][2];     // scale, and the powers of two that q was multiplied by, taken back
  uint32_t qf[NT][DIM / 8];
  int from = 0;             // first tile of the current piece
  int h0 = 0, gn = 0;       // the unit's first query head, and their number
  int done = 0;             // tiles whose copies are under way
  uint32_t put = ring_a, take = ring_a;  // the stages of the next tile to copy, to work on
  const uint32_t ring_end = ring_a + R::RING;
  auto issue = [&]() {
    if (done < n) {
      if (SPEAR_DCHECK(put >= ring_a && put + L::STAGE <= ring_end, p.hdr)) copy_tile(put);
      put = put + L::STAGE == ring_end ? ring_a : put + L::STAGE;
      advance<TILE>(p, in);
    }
    ++done;
    cp_commit();
  };
  // A new piece: its query heads' values, columns past them zero, as B fragments
  // in the order in which the codes' words come apart.
  auto begin_piece = [&]() {
    from = at.j;
    h0 = at.head * p.group + at.blk * 8 * NT;
    gn = min(8 * NT, p.group - at.blk * 8 * NT);
    constexpr int QB = KIND == SPEAR_KV_BF16 ? 8 : KIND == SPEAR_KV_INT8 ? 16 : (DIM >= 128 ? 32 : 16);
    // lane c holds dims [4 QB i + QB c, + QB) for each i
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const __nv_bfloat16* qr = p.q + at.b * p.ld_q + (long long)(h0 + nt * 8 + rho) * DIM;
#pragma unroll
      for (int i8 = 0; i8 < DIM / 32; ++i8) {
        const int d = (i8 / (QB / 8)) * 4 * QB + QB * cl + (i8 % (QB / 8)) * 8;
        uint4 w = make_uint4(0u, 0u, 0u, 0u);
        if (nt * 8 + rho < gn) w = *reinterpret_cast<const uint4*>(qr + d);
        uint32_t* f = qf[nt] + 4 * i8;
        f[0] = w.x, f[1] = w.y, f[2] = w.z, f[3] = w.w;
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int a = 0; a < MT; ++a)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[a][nt][e] = 0.f;
      q_scale[nt][0] = q_scale[nt][1] = p.scale;
      if constexpr (L::QUANT) {
        // to fp16, each head by the power of two that brings its largest value to
        // 2^14..2^15, so that nothing overflows and what is lost (of a sixteenth, for odd
        // nibbles) is under 2^-34 of it
        uint32_t m2 = 0u;
#pragma unroll
        for (int k = 0; k < DIM / 8; ++k) m2 = __vmaxu2(m2, qf[nt][k] & 0x7FFF7FFFu);
        uint32_t mag = max(m2 & 0xFFFFu, m2 >> 16);
        mag = max(mag, __shfl_xor_sync(ALL, mag, 1));
        mag = max(mag, __shfl_xor_sync(ALL, mag, 2));
        const int ex = mag >> 7;  // bf16's exponent field; 0: a zero row
        const int up = ex == 0 ? 127 : min(268 - ex, 253);
        const float f = __uint_as_float((uint32_t)up << 23);
        const float back = __uint_as_float((uint32_t)(254 - up) << 23);
        q_scale[nt][0] *= __shfl_sync(ALL, back, 8 * cl);
        q_scale[nt][1] *= __shfl_sync(ALL, back, 8 * cl + 4);
#pragma unroll
        for (int i8 = 0; i8 < DIM / 32; ++i8) {
          uint32_t* w = qf[nt] + 4 * i8;
          float x[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            x[2 * k] = __uint_as_float(w[k] << 16) * f;
            x[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u) * f;
          }
          if constexpr (KIND == SPEAR_KV_INT8) {  // bytes 0, 1 and 2, 3 of a word
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = pack_f16x2(x[2 * k], x[2 * k + 1]);
          } else {  // nibbles i and i + 4 of a word, the odd ones in sixteenths
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float part = k & 1 ? 0.0625f : 1.f;
              w[k] = pack_f16x2(x[k] * part, x[k + 4] * part);
            }
          }
        }
        const uint32_t even = KIND == SPEAR_KV_INT8 ? kLess128 : kLess8;
        const uint32_t less[4] = {even, even, kLess128, kLess128};
        float sq[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < DIM / 8; k += 2) mma<true>(sq, less, qf[nt][k], qf[nt][k + 1]);
        kfix[nt][0] = sq[0];
        kfix[nt][1] = sq[1];
      }
    }
  };
  // One tile; whole: every token of it is live.
  const int r0 = L::tok(rho), r1 = L::tok(rho + 8);
  auto work = [&](const uint32_t st, const int rows, auto whole) {
    constexpr bool WHOLE = decltype(whole)::value;
    // ---- scores: S[token][head] --------------------------------------------------------
    float s[TS][NT][4];  // scores
    [[maybe_unused]] float sv[TS][2];  // the values' scales of this lane's two tokens
    float top[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) top[nt][0] = top[nt][1] = -INFINITY;
#pragma unroll
    for (int b = 0; b < TS; ++b) {
      if (WHOLE || 16 * b < rows) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[b][nt][e] = L::QUANT ? kfix[nt][e & 1] : 0.f;
        const uint32_t ka = st + (16 * b + r0) * RB, kb = st + (16 * b + r1) * RB;
#pragma unroll
        for (int i4 = 0; i4 < L::KI; ++i4) {
          uint32_t x[L::KW], y[L::KW];
          if constexpr (L::KW == 4) {
            lds(ka + (((4 * i4 + cl) ^ L::xk(r0)) << 4), x);
            lds(kb + (((4 * i4 + cl) ^ L::xk(r1)) << 4), y);
          } else {
            lds(ka + cl * 4 * L::KW, x);
            lds(kb + cl * 4 * L::KW, y);
          }
          if constexpr (KIND == SPEAR_KV_BF16) {
#pragma unroll
            for (int k = 0; k < 4; k += 2) {
              const uint32_t a[4] = {x[k], y[k], x[k + 1], y[k + 1]};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma<false>(s[b][nt], a, qf[nt][4 * i4 + k], qf[nt][4 * i4 + k + 1]);
            }
          } else if constexpr (KIND == SPEAR_KV_INT8) {
#pragma unroll
            for (int k = 0; k < L::KW; ++k) {
              x[k] ^= kFlip, y[k] ^= kFlip;
              const uint32_t a[4] = {two_bytes<0x5150>(x[k]), two_bytes<0x5150>(y[k]), two_bytes<0x5352>(x[k]),
                                     two_bytes<0x5352>(y[k])};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma<true>(s[b][nt], a, qf[nt][2 * (L::KW * i4 + k)], qf[nt][2 * (L::KW * i4 + k) + 1]);
            }
          } else {
#pragma unroll
            for (int k = 0; k < L::KW; ++k)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t xh = h ? x[k] >> 8 : x[k], yh = h ? y[k] >> 8 : y[k];
                const uint32_t a[4] = {low4(xh), low4(yh), high4(xh), high4(yh)};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                  mma<true>(s[b][nt], a, qf[nt][4 * (L::KW * i4 + k) + 2 * h], qf[nt][4 * (L::KW * i4 + k) + 2 * h + 1]);
              }
          }
        }
        float f0 = 1.f, f1 = 1.f;
        if constexpr (L::QUANT) {
          const uint32_t sa = st + 2 * L::SIDE + 32 * b;
          f0 = lds_half(sa + 2 * r0) * kUnit;
          f1 = lds_half(sa + 2 * r1) * kUnit;
          sv[b][0] = lds_half(sa + 2 * TILE + 2 * r0);
          sv[b][1] = lds_half(sa + 2 * TILE + 2 * r1);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < EH; ++e) {
            s[b][nt][e] = s[b][nt][e] * f0 * q_scale[nt][e];
            s[b][nt][e + 2] = s[b][nt][e + 2] * f1 * q_scale[nt][e];
          }
        if (!WHOLE) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < EH; ++e) {
              if (16 * b + r0 >= rows) s[b][nt][e] = -INFINITY;
              if (16 * b + r1 >= rows) s[b][nt][e + 2] = -INFINITY;
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < EH; ++e) top[nt][e] = fmaxf(top[nt][e], fmaxf(s[b][nt][e], s[b][nt][e + 2]));
      }
    }
    // ---- the weights' reference m; what is there is scaled down where it moves -------------
    // m follows the maximum only once a weight is kSlack too large, which does no
    // harm: most tiles need neither the maximum over lanes nor new factors.
    bool above = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < EH; ++e) above |= top[nt][e] > m[nt][e] + kSlack;
    if (__any_sync(ALL, above)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float f[2];
#pragma unroll
        for (int e = 0; e < EH; ++e) {
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) top[nt][e] = fmaxf(top[nt][e], __shfl_xor_sync(ALL, top[nt][e], d));
          const float now = fmaxf(top[nt][e], m[nt][e]);
          f[e] = m[nt][e] == -INFINITY ? 0.f : exp2_(m[nt][e] - now);
          m[nt][e] = now;
          l[nt][e] *= f[e];
        }
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[a][nt][e] *= f[EH == 2 ? e & 1 : 0];
      }
    }
    float ref[NT][2];  // scores of -infinity alone leave m there: their weights are 0
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < EH; ++e) ref[nt][e] = m[nt][e] == -INFINITY ? 0.f : m[nt][e];
    // ---- weights, and O^T += V^T P -----------------------------------------------------------
#pragma unroll
    for (int b = 0; b < TS; ++b) {
      if (WHOLE || 16 * b < rows) {
        [[maybe_unused]] float f0 = 1.f, f1 = 1.f;
        if constexpr (L::QUANT) {
          f0 = sv[b][0], f1 = sv[b][1];
          if (!WHOLE) {  // scales of rows past the end may be anything
            if (16 * b + r0 >= rows) f0 = 0.f;
            if (16 * b + r1 >= rows) f1 = 0.f;
          }
        }
        uint32_t pb[NT][2], pl[NT][2];  // the weights' parts
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float e[4] = {};
#pragma unroll
          for (int k = 0; k < 4; k += 3 - EH) e[k] = exp2_(s[b][nt][k] - ref[nt][k & 1]);
          l[nt][0] += e[0] + e[2];
          if (EH == 2) l[nt][1] += e[1] + e[3];
          if constexpr (L::QUANT) e[0] *= f0, e[1] *= f0, e[2] *= f1, e[3] *= f1;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            split_bf16(e[2 * k], e[2 * k + 1], pb[nt][k], pl[nt][k]);
            if constexpr (EH == 1) pb[nt][k] |= pl[nt][k] << 16;  // the low part in the odd column
            else pl[nt][k] = movmatrix(pl[nt][k]);
            pb[nt][k] = movmatrix(pb[nt][k]);
          }
        }
        // The values' fragments a into the sums of 16 dims.  An infinite value counts
        // with the weights' high parts alone: their low parts may be 0 or negative,
        // and the sum NaN, where the formula's is infinite.
        auto add = [&](float (&o)[NT][4], const uint32_t (&a)[4], bool beyond = false) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma<false>(o[nt], a, pb[nt][0], pb[nt][1]);
          if constexpr (EH == 2) {
            uint32_t r[4] = {a[0], a[1], a[2], a[3]};
            if (KIND == SPEAR_KV_BF16 && beyond) {
#pragma unroll
              for (int k = 0; k < 4; ++k) r[k] = finite_part(r[k]);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma<false>(o[nt], r, pl[nt][0], pl[nt][1]);
          }
        };
        const uint32_t va = st + L::SIDE + 16 * b * RB;
        const int tk[4] = {L::tok(2 * cl), L::tok(2 * cl + 1), L::tok(2 * cl + 8), L::tok(2 * cl + 9)};
#pragma unroll
        for (int blk8 = 0; blk8 < DIM / (8 * L::VL); ++blk8) {
          uint32_t v[4][L::VW];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if constexpr (L::VW == 4) {
              lds(va + tk[k] * RB + (((8 * blk8 + rho) ^ L::xv(tk[k])) << 4), v[k]);
            } else if constexpr (L::VW == 2) {
              lds(va + tk[k] * RB + (((rho >> 1) ^ L::xv(tk[k])) << 4) + (rho & 1) * 8, v[k]);
            } else {
              lds(va + tk[k] * RB + rho * 4, v[k]);
            }
          }
          [[maybe_unused]] bool beyond = false;
          if constexpr (KIND == SPEAR_KV_BF16) beyond = __any_sync(ALL, any_beyond(v));
#pragma unroll
          for (int w = 0; w < L::VW; ++w) {
            // the same values of two tokens side by side: low halves, high halves
            const uint32_t lo01 = __byte_perm(v[0][w], v[1][w], 0x5410), hi01 = __byte_perm(v[0][w], v[1][w], 0x7632);
            const uint32_t lo89 = __byte_perm(v[2][w], v[3][w], 0x5410), hi89 = __byte_perm(v[2][w], v[3][w], 0x7632);
            constexpr int PER = L::VL / 2 / L::VW;  // products per word: 1, 2 or 4
            const int a0 = blk8 * (L::VL / 2) + w * PER;
            if constexpr (KIND == SPEAR_KV_BF16) {
              const uint32_t a[4] = {lo01, hi01, lo89, hi89};
              add(acc[a0], a, beyond);
            } else if constexpr (KIND == SPEAR_KV_INT8) {
              const uint32_t l01 = lo01 ^ kFlip, h01 = hi01 ^ kFlip, l89 = lo89 ^ kFlip, h89 = hi89 ^ kFlip;
              const uint32_t a[4] = {centred(two_bytes<0x5250>(l01), kOff128), centred(two_bytes<0x5351>(l01), kOff128),
                                     centred(two_bytes<0x5250>(l89), kOff128), centred(two_bytes<0x5351>(l89), kOff128)};
              const uint32_t c[4] = {centred(two_bytes<0x5250>(h01), kOff128), centred(two_bytes<0x5351>(h01), kOff128),
                                     centred(two_bytes<0x5250>(h89), kOff128), centred(two_bytes<0x5351>(h89), kOff128)};
              add(acc[a0], a);
              add(acc[a0 + 1], c);
            } else {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t l01 = h ? lo01 >> 8 : lo01, l89 = h ? lo89 >> 8 : lo89;
                const uint32_t h01 = h ? hi01 >> 8 : hi01, h89 = h ? hi89 >> 8 : hi89;
                const uint32_t a[4] = {centred(low4(l01), kOff8), centred(high4(l01), kOff128),
                                       centred(low4(l89), kOff8), centred(high4(l89), kOff128)};
                const uint32_t c[4] = {centred(low4(h01), kOff8), centred(high4(h01), kOff128),
                                       centred(low4(h89), kOff8), centred(high4(h89), kOff128)};
                add(acc[a0 + h], a);
                add(acc[a0 + 2 + h], c);
              }
            }
          }
        }
      }
    }
  };

#pragma unroll 1
  for (int i = 0; i < R::STAGES - 1; ++i) issue();
  bool fresh = true;
  for (int i = 0; i < n; ++i) {
    if (fresh) begin_piece();
    cp_wait<R::STAGES - 2>();
    __syncwarp();  // tile i is in, and every lane is through with tile i - 1
    issue();
    const int rows = at.len - at.j * TILE;  // live tokens from the tile's first on
    if (rows >= TILE) work(take, rows, std::true_type{});
    else work(take, rows, std::false_type{});
    take = take + L::STAGE == ring_end ? ring_a : take + L::STAGE;
    // ---- the end of the unit or of the run ------------------------------------------------
    // What runs once or twice a launch is kept short rather than fast, here and
    // below: lines of code that the stream through L2 has pushed out take long to come.
    fresh = at.j + 1 == at.nt;
    if (fresh || i + 1 == n) {
      if constexpr (EH == 1) {  // the parts' products
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
          for (int e = 0; e < 4; e += 2) acc[a][0][e] += acc[a][0][e + 1];
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < EH; ++e)
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) l[nt][e] += __shfl_xor_sync(ALL, l[nt][e], d);
      if (fresh && from == 0) {  // the whole unit: out with it
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < EH; ++e) {
            const int h = nt * 8 + 2 * cl + e;
            if (h < gn && SPEAR_DCHECK(at.b < p.n_seqs && h0 + h < p.heads, p.hdr)) {
              const float even = (L::QUANT ? kValue : 1.f) / l[nt][e], odd = KIND == SPEAR_KV_INT4 ? 0.0625f * even : even;
              __nv_bfloat16* o = p.out + at.b * p.ld_out + (long long)(h0 + h) * DIM;
#pragma unroll
              for (int a = 0; a < MT; a += 4) {
                const int d = (a / (L::VL / 2)) * 8 * L::VL + rho * L::VL + 2 * (a % (L::VL / 2));
                uint4 w;
                w.x = pack_bf16x2(acc[a][nt][e] * even, acc[a][nt][e + 2] * odd);
                w.y = pack_bf16x2(acc[a + 1][nt][e] * even, acc[a + 1][nt][e + 2] * odd);
                w.z = pack_bf16x2(acc[a + 2][nt][e] * even, acc[a + 2][nt][e + 2] * odd);
                w.w = pack_bf16x2(acc[a + 3][nt][e] * even, acc[a + 3][nt][e + 2] * odd);
                *reinterpret_cast<uint4*>(o + d) = w;
              }
              if (p.lse && rho == 0)
                p.lse[(long long)at.b * p.heads + h0 + h] = (m[nt][e] + log2f(l[nt][e])) * 0.6931471805599453f;
            }
          }
      } else {
        if (!fresh) {
          // every copy is in and read: the ring is this piece's place
          cp_wait<0>();
          __syncwarp();
        }
        float* dst = fresh ? first_piece : last_piece;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < EH; ++e) {
            const int h = nt * 8 + 2 * cl + e;
#pragma unroll
            for (int a = 0; a < MT; ++a) {
              const int d = (a / (L::VL / 2)) * 8 * L::VL + rho * L::VL + 2 * (a % (L::VL / 2));
              *reinterpret_cast<float2*>(dst + h * DIM + d) = make_float2(acc[a][nt][e], acc[a][nt][e + 2]);
            }
            if (rho == 0) {
              dst[8 * NT * DIM + h] = m[nt][e];
              dst[8 * NT * DIM + 8 * NT + h] = l[nt][e];
            }
          }
        if (lane == 0) pieces[2 * warp + !fresh] = {start, at.nt, from, at.j + 1, at.b, h0, gn};
      }
    }
    if (fresh) start += at.nt + 1;
    advance<TILE>(p, at);
  }
  cp_wait<0>();
  __syncthreads();

  // ---- join the pieces of each unit -----------------------------------------------------------
  constexpr int CH = (DIM + 127) / 128;      // 128-value parts of a head: one per warp and step
  constexpr int LD = DIM >= 128 ? 128 : DIM;  // values of such a part
  // Of a piece of maximum pm where mx is the largest so far; its sums are
  // 0 where all its scores are -infinity, and 0 / 0 follows where all pieces' are.
  auto weight = [&](float pm, float mx) { return pm == -INFINITY ? 0.f : exp2_(pm - mx); };
  // Part `item` (head, part) of a unit's pieces joined: their common maximum
  // mx and sum, and LD values o of the output, one float4 per lane.  It goes to the
  // output, or to `part` where pieces of other CTAs are still to come.
  auto put_item = [&](const Piece& pc, int item, float mx, float sum, float4 o, float* part) {
    const int h = item / CH, d = (item % CH) * 128 + 4 * lane;
    if (4 * lane >= LD) return;
    if (part) {
      if (!SPEAR_DCHECK(part >= p.parts && part + R::PIECE <= p.parts + (size_t)p.ctas * 2 * R::PIECE, p.hdr)) return;
      __stcg(reinterpret_cast<float4*>(part + h * DIM + d), o);
      if (d == 0) {
        __stcg(part + 8 * NT * DIM + h, mx);
        __stcg(part + 8 * NT * DIM + 8 * NT + h, sum);
      }
    } else if (SPEAR_DCHECK(pc.b < p.n_seqs && pc.h0 + h < p.heads, p.hdr)) {
      const float inv = (L::QUANT ? kValue : 1.f) / sum;
      if constexpr (KIND == SPEAR_KV_INT4) o.y *= 0.0625f, o.w *= 0.0625f;  // odd dims, from bits 4-7
      *reinterpret_cast<uint2*>(p.out + pc.b * p.ld_out + (long long)(pc.h0 + h) * DIM + d) =
          make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
      if (p.lse && d == 0) p.lse[(long long)pc.b * p.heads + pc.h0 + h] = (mx + log2f(sum)) * 0.6931471805599453f;
    }
  };
  // Pieces `set` of this CTA: lane k has piece k's maximum and sum.
  auto join_here = [&](const Piece& pc, int item, unsigned set, float* part) {
    const int h = item / CH, d = (item % CH) * 128 + 4 * lane;
    if (h >= pc.num) return;
    auto piece_of = [&](int e) {
      uint8_t* r = smem + (size_t)(e >> 1) * (R::RING + R::PIECE * 4);
      return reinterpret_cast<const float*>(e & 1 ? r : r + R::RING);
    };
    float pm = -INFINITY, w = 0.f, sum = 0.f;
    const bool has = set >> lane & 1;
    if (has) {
      const float* f = piece_of(lane) + 8 * NT * DIM + h;
      pm = f[0];
      sum = f[8 * NT];
    }
    float mx = pm;
#pragma unroll
    for (int e = 8; e > 0; e >>= 1) mx = fmaxf(mx, __shfl_xor_sync(ALL, mx, e));  // 2 W <= 16 pieces
    mx = __shfl_sync(ALL, mx, 0);
    if (has) w = weight(pm, mx);
    sum *= w;
#pragma unroll
    for (int e = 8; e > 0; e >>= 1) sum += __shfl_xor_sync(ALL, sum, e);
    sum = __shfl_sync(ALL, sum, 0);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (; set; set &= set - 1) {
      const int k = __ffs(set) - 1;
      const float wk = __shfl_sync(ALL, w, k);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (4 * lane < LD) v = *reinterpret_cast<const float4*>(piece_of(k) + h * DIM + d);
      o.x = fmaf(wk, v.x, o.x);
      o.y = fmaf(wk, v.y, o.y);
      o.z = fmaf(wk, v.z, o.z);
      o.w = fmaf(wk, v.w, o.w);
    }
    put_item(pc, item, mx, sum, o, part);
  };
  // Where CTA c of a unit that begins in CTA c0 has its part: the first on its far side.
  auto part_of = [&](int c, int c0) { return p.parts + ((size_t)c * 2 + (c == c0)) * R::PIECE; };
  // The parts of `count` CTAs, `every` apart from `first` on, read past this SM's L1, to
  // the output or to `part`: each warp has up to I items, of STEP parts at a time, all
  // asked for before any is used.
  auto join_parts = [&](const Piece& pc, int c0, int first, int every, int count, float* part) {
    constexpr int I = (8 * NT * CH + W - 1) / W, STEP = 16 / I;
    float mx[I], sum[I];
    float4 o[I];
#pragma unroll
    for (int c = 0; c < I; ++c) mx[c] = -INFINITY, sum[c] = 0.f, o[c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int k0 = 0; k0 < count; k0 += STEP) {
      float pm[I][STEP], pl[I][STEP];
      float4 pv[I][STEP];
#pragma unroll
      for (int k = 0; k < STEP; ++k) {
        const float* f = part_of(first + (k0 + k) * every, c0);
#pragma unroll
        for (int c = 0; c < I; ++c) {
          const int item = warp + c * W, h = item / CH, d = (item % CH) * 128 + 4 * lane;
          pm[c][k] = -INFINITY;
          pl[c][k] = 0.f;
          pv[c][k] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (k0 + k < count && h < pc.num) {
            pm[c][k] = __ldcg(f + 8 * NT * DIM + h);
            pl[c][k] = __ldcg(f + 8 * NT * DIM + 8 * NT + h);
            if (4 * lane < LD) pv[c][k] = __ldcg(reinterpret_cast<const float4*>(f + h * DIM + d));
          }
        }
      }
#pragma unroll
      for (int c = 0; c < I; ++c) {
        float top = mx[c];
#pragma unroll
        for (int k = 0; k < STEP; ++k) top = fmaxf(top, pm[c][k]);
        const float keep = mx[c] == -INFINITY ? 0.f : exp2_(mx[c] - top);
        mx[c] = top;
        sum[c] *= keep;
        o[c].x *= keep, o[c].y *= keep, o[c].z *= keep, o[c].w *= keep;
#pragma unroll
        for (int k = 0; k < STEP; ++k) {
          const float w = k0 + k < count ? weight(pm[c][k], top) : 0.f;
          sum[c] = fmaf(w, pl[c][k], sum[c]);
          o[c].x = fmaf(w, pv[c][k].x, o[c].x);
          o[c].y = fmaf(w, pv[c][k].y, o[c].y);
          o[c].z = fmaf(w, pv[c][k].z, o[c].z);
          o[c].w = fmaf(w, pv[c][k].w, o[c].w);
        }
      }
    }
    if (part) __syncthreads();  // it may be one of those just read
#pragma unroll
    for (int c = 0; c < I; ++c)
      if ((warp + c * W) / CH < pc.num) put_item(pc, warp + c * W, mx[c], sum[c], o[c], part);
  };
  // Lane i of every warp looks at piece i; a unit's pieces are neighbours among those
  // that are there.  heads: the first piece of each unit.
  const bool mine_there = lane < 2 * W && pieces[lane].to > 0;
  const unsigned there = __ballot_sync(ALL, mine_there), below = there & ((1u << lane) - 1u);
  unsigned heads =
      __ballot_sync(ALL, mine_there && (!below || pieces[31 - __clz(below)].start != pieces[lane].start));
  const int items = min(p.group, 8 * NT) * CH;
  int open[2] = {-1, -1};  // first pieces of the units that come from another CTA, go on in one
  for (int at_item = warp; heads; heads &= heads - 1) {
    const int k = __ffs(heads) - 1;
    const unsigned later = heads & (heads - 1);
    const unsigned set = there & ~((1u << k) - 1u) & (later ? (1u << (__ffs(later) - 1)) - 1u : ~0u);
    const int last = 31 - __clz(set);
    const bool starts = pieces[k].from == 0, ends = pieces[last].to == pieces[k].nt;
    float* part = nullptr;
    if (!(starts && ends)) {
      open[starts] = k;
      part = p.parts + ((size_t)blockIdx.x * 2 + starts) * R::PIECE;
    }
    // the items of all units are dealt to the warps in turn
    for (; at_item < items; at_item += W) join_here(pieces[k], at_item, set, part);
    at_item -= items;
  }
  if (open[0] < 0 && open[1] < 0) return;
  // Who counts last at a unit's ticket, which is then back at zero, joins its parts;
  // of many, first those of its group, to the place of the group's first.  Thread 0
  // sees to the one unit, thread 1 to the other.  Every thread's parts are ordered
  // before the count by the barrier and its release, and those of others are read
  // after its acquire.
  Job job = {};
  int* ticket = nullptr;
  int count = 0;
  if (tid < 2 && open[tid] >= 0) {
    const Piece& pc = pieces[open[tid]];
    job.c0 = job.first = cut.owner(pc.start + 1);
    job.every = 1;
    job.n = count = cut.owner(pc.start + pc.nt) - job.c0 + 1;
    ticket = p.tickets + job.c0;
    if (count > kRadix) {
      job.group = true;
      job.first += (int)(blockIdx.x - job.c0) / kRadix * kRadix;
      job.n = min(kRadix, job.c0 + count - job.first);
      // a unit's last CTA may be the first of another's: each counts on its part's side
      ticket = p.tickets + p.ctas + 2 * job.first + (job.first == job.c0);
    }
    if (!SPEAR_DCHECK(job.c0 >= 0 && job.c0 + count <= (int)ctas, p.hdr)) ticket = nullptr;
  }
#pragma unroll 1
  for (bool more = true; more;) {
    __syncthreads();
    if (tid < 2) {
      job.mine = false;
      if (ticket) {
        int old;
        asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(old) : "l"(ticket) : "memory");
        job.mine = old == job.n - 1;
        if (job.mine) *ticket = 0;
      }
      jobs[tid] = job;
      if (!job.mine || !job.group) {
        ticket = nullptr;
      } else {  // then the groups' parts
        job.group = false;
        job.first = job.c0;
        job.every = kRadix;
        job.n = (count + kRadix - 1) / kRadix;
        ticket = p.tickets + job.c0;
      }
    }
    __syncthreads();
    more = false;
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {
      const Job j = jobs[side];
      if (!j.mine) continue;
      join_parts(pieces[open[side]], j.c0, j.first, j.every, j.n, j.group ? part_of(j.first, j.c0) : nullptr);
      more |= j.group;
    }
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
struct AttnPlan {
  int nt, blocks;
  int piece;  // floats of a part, Room::PIECE, at most
  int ctas;   // at most
};

// tokens: of all sequences, at most.  Groups of more than 8 query heads go through
// two products side by side, which read a tile once, where there are tiles enough;
// else as units of 8 each, of which twice as many warps run and join smaller parts
// (heads 48/4 of 128, sequences to 4096; int8: 64 of them 55.9 us, 65.4 as units of
// 8, 32 of them 37.3, 39.4, 16 of them 24.6, 22.0; bf16: 64 of them 63.2, 88.8, 16 of
// them 27.5, 26.6, 8 of them 23.5, 19.3; int4: 47.6, 58.0, and 23.3, 20.4).  The host does
// not know the lengths, so the table's room counts: short sequences under a wide
// table get the form that is slower for them (int8, 16 of up to 512 tokens: 16.5 us
// under a table for 65,536, 12.0 under one for 512).  256-wide heads have no
// registers for two products: their groups past 8 always read the cache again (bf16,
// 8 of up to 32,768, 2 kv heads: 55.5 us with 8 heads each, 77.5 with 16).
static AttnPlan plan_attn(const KvView& c, int n_q_heads, long long tokens) {
  AttnPlan a;
  const int group = n_q_heads / c.heads;
  const bool may_pair = group > 8 && c.dim < 256;
  a.nt = may_pair && tokens * c.heads > 2560LL * device_sm_count() ? 2 : 1;
  a.blocks = (group + 8 * a.nt - 1) / (8 * a.nt);
  a.piece = (8 * (may_pair ? 2 : 1) * (c.dim + 2) + 3) / 4 * 4;
  a.ctas = device_sm_count() * attn_per_sm(c.kind, c.dim);
  return a;
}

static size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

// Header and counters, which take the same place for every cache, so that calls for
// caches of several shapes can take turns in one workspace.
static size_t attn_ws_parts() { return kWsHeaderBytes + up256(3 * 2 * (size_t)device_sm_count() * sizeof(int)); }
static size_t attn_ws_bytes(const AttnPlan& a) {
  return attn_ws_parts() + up256((size_t)a.ctas * 2 * a.piece * sizeof(float));
}

template <int KIND, int DIM, int NT, int EH>
static cudaError_t launch_attn(AttnArgs& a, const AttnPlan& pl, cudaStream_t st) {
  using L = Lay<KIND, DIM>;
  using R = Room<KIND, DIM, NT>;
  constexpr int W = R::W;
  auto* k = attn_kernel<KIND, DIM, NT, EH, W, R::PER_SM>;
  static std::atomic<uint64_t> ready{0};  // devices whose limit is raised
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, R::BYTES);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  // no more CTAs than the longest possible line gives work to
  const long long tiles = (long long)a.c.heads * a.blocks * a.n_seqs * ((a.max_len + L::TILE - 1) / L::TILE + 1);
  if (tiles >> 32) return cudaErrorInvalidConfiguration;  // refused before
  const long long need = (tiles + (long long)kMinTiles * W - 1) / ((long long)kMinTiles * W);
  const long long all_units = (long long)a.c.heads * a.blocks * a.n_seqs;
  const long long most = need > all_units ? need : all_units;
  const int grid = (int)(most < pl.ctas ? most : pl.ctas);
  return launch_after(k, dim3(grid), W * 32, R::BYTES, st, a);
}

}  // namespace spear

using namespace spear;

extern "C" size_t spear_attn_workspace_bytes(const spear_kv_cache* cache, int n_q_heads) {
  KvView c;
  if (check_kv_cache(cache, &c) != SPEAR_OK || n_q_heads < 1 || n_q_heads > 1024 || n_q_heads % c.heads) return 0;
  return attn_ws_bytes(plan_attn(c, n_q_heads, 0));
}

extern "C" int spear_attn_decode(const spear_kv_cache* cache, const uint16_t* q, long long ld_q, int n_seqs,
                                 int n_q_heads, const int* page_table, int max_pages, int ld_table,
                                 const int* seq_lens, float scale, uint16_t* out, long long ld_out, float* lse,
                                 void* ws, size_t ws_bytes, void* stream) {
  TraceRange trace_("spear_attn_decode");
  clear_error();
  AttnArgs a = {};
  const int rc = check_kv_cache(cache, &a.c);
  if (rc) return rc;
  if (n_q_heads < 1 || n_q_heads > 1024 || n_q_heads % a.c.heads)
    return set_error(SPEAR_ERR_UNSUPPORTED_SHAPE, "n_q_heads=%d: a multiple of the cache's %d heads, at most 1024",
                     n_q_heads, a.c.heads);
  if (n_seqs < 0 || n_seqs > kMaxSeqs) return set_error(SPEAR_ERR_UNSUPPORTED_SHAPE, "n_seqs=%d: must be 0 to 4096", n_seqs);
  if (n_seqs == 0) return SPEAR_OK;
  if (!q || !page_table || !seq_lens || !out || !ws) return set_error(SPEAR_ERR_INVALID_ARG, "NULL pointer");
  if (!(fabsf(scale * kLog2e) < INFINITY))
    return set_error(SPEAR_ERR_INVALID_ARG, "scale=%g: it and its product with log2(e) must be finite", scale);
  if (max_pages < 1 || ld_table < max_pages)
    return set_error(SPEAR_ERR_INVALID_ARG, "max_pages=%d ld_table=%d: 1 <= max_pages <= ld_table", max_pages, ld_table);
  if ((long long)max_pages * a.c.page_size > 0x7fff0000LL)
    return set_error(SPEAR_ERR_UNSUPPORTED_SHAPE, "max_pages=%d: a sequence holds less than 2^31 - 2^16 tokens", max_pages);
  if ((long long)n_seqs * max_pages * (a.c.page_size / 16) * n_q_heads >> 31)
    return set_error(SPEAR_ERR_UNSUPPORTED_SHAPE,
                     "n_seqs=%d max_pages=%d: sequences x tokens x query heads must be under 2^35", n_seqs, max_pages);
  const long long row = (long long)n_q_heads * a.c.dim;
  if (ld_q < row || ld_out < row || ld_q % 8 || ld_out % 8)
    return set_error(SPEAR_ERR_INVALID_ARG, "ld_q=%lld ld_out=%lld: multiples of 8 of at least %lld", ld_q, ld_out, row);
  if (!ptr_aligned16(q) || !ptr_aligned16(out) || !ptr_aligned16(ws))
    return set_error(SPEAR_ERR_ALIGNMENT, "q, out and ws must be 16-byte aligned");
  for (const void* p : {(const void*)page_table, (const void*)seq_lens, (const void*)lse})
    if (reinterpret_cast<uintptr_t>(p) & 3u)
      return set_error(SPEAR_ERR_ALIGNMENT, "page_table, seq_lens and lse must be 4-byte aligned");
  const uintptr_t q_bytes = ((n_seqs - 1) * ld_q + row) * 2, out_bytes = ((n_seqs - 1) * ld_out + row) * 2;
  const uintptr_t table_bytes = ((n_seqs - 1LL) * ld_table + max_pages) * 4, lens_bytes = n_seqs * 4LL;
  const uintptr_t lse_bytes = (long long)n_seqs * n_q_heads * 4;
  if (buffers_meet(lse, lse_bytes, q, q_bytes) || buffers_meet(lse, lse_bytes, out, out_bytes))
    return set_error(SPEAR_ERR_INVALID_ARG, "lse and q or out overlap");
  if (buffers_meet(lse, lse_bytes, page_table, table_bytes) || buffers_meet(lse, lse_bytes, seq_lens, lens_bytes) ||
      buffers_meet(out, out_bytes, page_table, table_bytes) || buffers_meet(out, out_bytes, seq_lens, lens_bytes))
    return set_error(SPEAR_ERR_INVALID_ARG, "an output and page_table or seq_lens overlap");
  // q and out may be column ranges of the same rows, and share nothing else
  if (buffers_meet(q, q_bytes, out, out_bytes)) {
    const long long apart = (long long)(reinterpret_cast<uintptr_t>(out) - reinterpret_cast<uintptr_t>(q)) / 2;
    const long long column = (apart % ld_q + ld_q) % ld_q;
    if (n_seqs == 1 || ld_q != ld_out || column < row || column + row > ld_q)
      return set_error(SPEAR_ERR_INVALID_ARG, "q and out overlap");
  }
  const AttnPlan pl = plan_attn(a.c, n_q_heads, (long long)n_seqs * max_pages * a.c.page_size);
  const size_t need = attn_ws_bytes(pl);
  if (ws_bytes < need) return set_error(SPEAR_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", ws_bytes, need);
  a.q = reinterpret_cast<const __nv_bfloat16*>(q);
  a.out = reinterpret_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.table = page_table;
  a.lens = seq_lens;
  a.ld_q = ld_q;
  a.ld_out = ld_out;
  a.ld_table = ld_table;
  a.max_len = max_pages * a.c.page_size;
  a.n_seqs = n_seqs;
  a.heads = n_q_heads;
  a.group = n_q_heads / a.c.heads;
  a.blocks = pl.blocks;
  a.scale = scale * kLog2e;
  uint8_t* w = static_cast<uint8_t*>(ws);
  a.hdr = reinterpret_cast<WsHeader*>(w);
  a.tickets = reinterpret_cast<int*>(w + kWsHeaderBytes);
  a.parts = reinterpret_cast<float*>(w + attn_ws_parts());
  a.ctas = pl.ctas;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaErrorInvalidValue;
  for_kind_dim(a.c.kind, a.c.dim, [&](auto kc, auto dc) {
    if constexpr (dc.value < 256)
      if (pl.nt == 2) {
        e = launch_attn<kc.value, dc.value, 2, 2>(a, pl, st);
        return;
      }
    // One query head per kv head: a lane's second column is none, its softmax is left
    // out, and the second products too (int4, 32 x 4099, 32 heads: 65.8 us, 69.0 with
    // the products).  bf16 waits for HBM.
    if constexpr (kc.value != SPEAR_KV_BF16)
      if (a.group == 1) {
        e = launch_attn<kc.value, dc.value, 1, 1>(a, pl, st);
        return;
      }
    e = launch_attn<kc.value, dc.value, 1, 2>(a, pl, st);
  });
  return e == cudaSuccess ? SPEAR_OK : set_cuda_error("attention launch", e);
}
