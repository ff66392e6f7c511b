// The gradient of the joint attention (Ideogram 4 deep dive, section 4-2: one sequence, one
// bidirectional self-attention), the probabilities recomputed from q, k and the row log-sum-exps:
//   P = exp(q k^T / sqrt(hd) - lse)         delta_q = sum_c dO_qc O_qc
//   dV = P^T dO     dP = dO V^T     dS = P o (dP - delta) / sqrt(hd)     dQ = dS K     dK = dS^T Q
// Two launches:
//   bwd_prep_kernel  delta and the row log-sum-exps in log2 units, padded to whole blocks of 128
//                    rows, and what the passes need to know of the data (see below)
//   bwd_kernel       the key pass (dK, dV: 256 keys per CTA pair, over all query blocks), then the query
//                    pass (dQ: 256 queries per CTA pair, over all key blocks)
// S and dP are computed in both passes, seven products instead of five: dQ is summed over
// the keys and dK, dV over the queries, and a single pass would have to add one of them up in
// global memory, by fp32 atomics (whose order changes the result from run to run) or through
// S / 128 partial copies of it (more HBM time than the two extra products take).
//
// Padded batches: element b's tokens are its first n_b rows; the other rows take no part and their
// gradients are zero whatever they hold, infinities and NaN included.  A masked probability of
// zero times a NaN row would still be NaN inside the tensor core, so the block in which the
// tokens end is read from zero-padded copies (tails) that bwd_prep_kernel makes.
//
// Roundings.  S, dP and all sums are fp32.  P and dS are rounded once to the inputs' 16-bit format,
// the operand type of the products they enter.  In f16 they are scaled by powers of two first, since
// typical values (P ~ 1/S, dS smaller still) sit in or below f16's subnormal range: P by 2^15
// (P <= 1), dS by a sigma, both undone on the fp32 accumulators.  With A the Euclidean norm of a row of dO
// over one head's channels and B = max_k |V_k|, |dP - delta| <= 2 A B in that row, so
// sigma = 2^floor(14 - log2(2 A B)) keeps its |dS| below 2^15.  The query pass, whose accumulator rows
// are queries, takes each row's own A: a row 2^24 times smaller than another keeps its 11 bits.  The key pass
// sums over the queries and takes the largest A of the head: each dS there is held to within 2^-38 of the
// head's largest 2 A B (half of f16's last step, 2^-25, over 2^13) or to 11 bits, whichever is coarser.
#include "common.cuh"
#include "pipeline.cuh"
#include "train.h"

namespace jab {
namespace abwd {

constexpr int T = 128;  // rows of an own tile per CTA
constexpr int TMEM_COLS = 512;
constexpr float LOG2E = 1.4426950408889634f;
constexpr float P_SHIFT = 15.f;  // f16: P is held as 2^15 P

// The shape of one pass: blocks of R rows of the streamed axis, COLS of them per elementwise thread (a
// warp works on a 32 x COLS piece), SLOTS blocks of operands in flight.
// OUT columns of an accumulator are staged per warp for the store; VECS slots of row vectors.
// dkv's blocks are the largest whose S^T, dP^T, P^T and dS^T (3 R columns) fit TMEM beside dV and dK.
template <int HD>
struct DkvShape {
  static constexpr int R = 80, COLS = 16, SLOTS = 3, CUTS_B = 2, OUT = 32, VECS = 5;
};
template <>
struct DkvShape<64> {
  static constexpr int R = 128, COLS = 32, SLOTS = 3, CUTS_B = 2, OUT = 32, VECS = 5;
};
struct DqShape {
  static constexpr int R = 128, COLS = 32, SLOTS = 3, CUTS_B = 1, OUT = 16, VECS = 0;
};

__host__ __device__ inline int blocks_of(int seq) { return (seq + T - 1) / T; }

// Per (b, h), nblk = the blocks of 128 rows and one more (blocks of any R <= 128 rows end inside it):
// nlse2 / ndelta / rows2 [B, H, nblk * 128], -log2(e) lse, -delta and (f16 only) |dO_q|^2; norms2
// [B, H, nblk]: the block's max |dO_q|^2 and max |V_k|^2 (f16 only); tails: zero-padded copies
// [3: q, k, dO][B, 128, H hd] of the
// block in which the tokens end.
struct Workspace {
  float* nlse2;
  float* ndelta;
  float* rows2;
  float2* norms2;
  uint16_t* tails;
  size_t bytes;
};

static size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

static Workspace carve(void* base, int batch, int seq, int n_heads, int head_dim) {
  Workspace w{};
  const size_t bh = static_cast<size_t>(batch) * n_heads, nblk = blocks_of(seq) + 1;
  const size_t vec = align256(bh * nblk * T * 4), nrm = align256(bh * nblk * 8);
  const size_t tail = align256(static_cast<size_t>(batch) * T * n_heads * head_dim * 2 * 3);
  uint8_t* b = static_cast<uint8_t*>(base);
  w.nlse2 = reinterpret_cast<float*>(b);
  w.ndelta = reinterpret_cast<float*>(b + vec);
  w.rows2 = reinterpret_cast<float*>(b + 2 * vec);
  w.norms2 = reinterpret_cast<float2*>(b + 3 * vec);
  w.tails = reinterpret_cast<uint16_t*>(b + 3 * vec + nrm);
  w.bytes = 3 * vec + nrm + tail;
  return w;
}

__device__ __forceinline__ int tokens_of(const int32_t* key_lens, int b, int seq) {
  return key_lens == nullptr ? seq : min(max(key_lens[b], 0), seq);
}
// The element's last block of `rows` rows is read from its tail copy.
__device__ __forceinline__ bool has_tail(int n, int seq, int rows) { return n < seq && n % rows != 0; }

struct PrepArgs {
  const uint16_t *q, *k, *v, *o, *dout;
  int64_t ldq, ldk, ldv;
  const float* lse;
  const int32_t* key_lens;
  float *nlse2, *ndelta, *rows2;
  float2* norms2;
  uint16_t* tails;
  int batch, seq, n_heads;
};

// One CTA per (block of 128 rows, head, element); HD / 8 lanes per row.  HBM-bound: reads O and dO
// (f16: and V) once.  4608 tokens x 32 heads of 128, L2 cold: bf16 19.5 us (75 MB, 3.9 TB/s), f16
// 26.4 us (113 MB, 4.3 TB/s), 2-3 % of the whole gradient.  Latency counts in the small calls, so each
// thread has few rows and loads two of them at a time: 1100 tokens x 16 heads 6.7 us and 80 tokens x 4
// heads 3.8, against 9.2 and 5.2 with 256 threads; one row at a time 17.8 / 25.0 / 7.7 / 4.4 us; with all
// rows' loads of 256 threads in flight the registers cost the large f16 call 36 us.
constexpr int PREP_THREADS = 512;
template <int HD, int F>
__global__ void __launch_bounds__(PREP_THREADS, 3) bwd_prep_kernel(const PrepArgs a) {
  constexpr int LANES = HD / 8;
  constexpr int ROWS = PREP_THREADS / LANES;
  constexpr int PASSES = T / ROWS;
  __shared__ float2 red[PREP_THREADS / 32];
  pdl_wait_then_release();
  const int blk = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int nblk = gridDim.x;
  const int n = tokens_of(a.key_lens, b, a.seq);
  const int d = a.n_heads * HD;
  const int c = static_cast<int>(threadIdx.x) % LANES, r0 = static_cast<int>(threadIdx.x) / LANES;
  const int64_t bh = static_cast<int64_t>(b) * a.n_heads + h;
  float* nlse2 = a.nlse2 + (bh * nblk + blk) * T;
  float* ndelta = a.ndelta + (bh * nblk + blk) * T;
  float* rows2 = a.rows2 + (bh * nblk + blk) * T;
  float mdo = 0.f, mv = 0.f;
  // rows that take no part read the element's first row (a block past the tokens reads none)
  constexpr int CHUNK = 2;
  static_assert(PASSES % CHUNK == 0, "whole chunks");
  const bool any = blk * T < n;
#pragma unroll 1
  for (int p0 = 0; p0 < PASSES; p0 += CHUNK) {
    uint4 ro[CHUNK], rg[CHUNK], rv[F == FMT_F16 ? CHUNK : 1];
    if (any) {
#pragma unroll
      for (int p = 0; p < CHUNK; ++p) {
        const int row = blk * T + (p0 + p) * ROWS + r0;
        const int64_t at = static_cast<int64_t>(b) * a.seq + (row < n ? row : 0);
        ro[p] = reinterpret_cast<const uint4*>(a.o + at * d + h * HD)[c];
        rg[p] = reinterpret_cast<const uint4*>(a.dout + at * d + h * HD)[c];
        if constexpr (F == FMT_F16) rv[p] = reinterpret_cast<const uint4*>(a.v + at * a.ldv + h * HD)[c];
      }
    }
#pragma unroll
    for (int p = 0; p < CHUNK; ++p) {
      const int r = (p0 + p) * ROWS + r0;
      const int row = blk * T + r;
      float dot = 0.f, sdo = 0.f, sv = 0.f;
      if (row < n) {
        float o[8], g[8];
        load8<F>(&ro[p], 0, o);
        load8<F>(&rg[p], 0, g);
#pragma unroll
        for (int k = 0; k < 8; ++k) dot = fmaf(o[k], g[k], dot);
        if constexpr (F == FMT_F16) {
          float v[8];
          load8<F>(&rv[p], 0, v);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            sdo = fmaf(g[k], g[k], sdo);
            sv = fmaf(v[k], v[k], sv);
          }
        }
      }
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1) {
        dot += __shfl_xor_sync(0xffffffffu, dot, o);
        if constexpr (F == FMT_F16) {
          sdo += __shfl_xor_sync(0xffffffffu, sdo, o);
          sv += __shfl_xor_sync(0xffffffffu, sv, o);
        }
      }
      mdo = fmaxf(mdo, sdo);
      mv = fmaxf(mv, sv);
      if (c == 0) {
        // rows that take no part: exp2(s - inf) = 0
        ndelta[r] = -dot;
        if constexpr (F == FMT_F16) rows2[r] = sdo;
        nlse2[r] = row < n ? (F == FMT_F16 ? P_SHIFT : 0.f) - a.lse[bh * a.seq + row] * LOG2E : -INFINITY;
      }
    }
  }
  if constexpr (F == FMT_F16) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      mdo = fmaxf(mdo, __shfl_xor_sync(0xffffffffu, mdo, o));
      mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, o));
    }
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(mdo, mv);
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < PREP_THREADS / 32; ++w) {
        mdo = fmaxf(mdo, red[w].x);
        mv = fmaxf(mv, red[w].y);
      }
      a.norms2[bh * nblk + blk] = make_float2(mdo, mv);
    }
  }
  // k: the block in which the tokens end in dq's blocks; q and dO: in dkv's
  constexpr int RK = DqShape::R, RQ = DkvShape<HD>::R;
  const int k0 = n / RK * RK, q0 = n / RQ * RQ;
  auto reaches = [&](int row0, int rows) { return blk * T < row0 + rows && blk * T + T > row0; };
  const bool tk = has_tail(n, a.seq, RK) && reaches(k0, RK), tq = has_tail(n, a.seq, RQ) && reaches(q0, RQ);
  if (tk || tq) {
    const size_t one = static_cast<size_t>(a.batch) * T * d;
    for (int p = 0; p < PASSES; ++p) {
      const int row = blk * T + p * ROWS + r0;
      const int64_t at = static_cast<int64_t>(b) * a.seq + row;
      auto put = [&](const uint16_t* src, int64_t ld, int which, int dst_row) {
        const uint4 x = row < n ? reinterpret_cast<const uint4*>(src + at * ld + h * HD)[c] : make_uint4(0u, 0u, 0u, 0u);
        reinterpret_cast<uint4*>(a.tails + which * one + (static_cast<size_t>(b) * T + dst_row) * d + h * HD)[c] = x;
      };
      if (tk && row >= k0 && row < k0 + RK) put(a.k, a.ldk, 1, row - k0);
      if (tq && row >= q0 && row < q0 + RQ) {
        put(a.q, a.ldq, 0, row - q0);
        put(a.dout, d, 2, row - q0);
      }
    }
  }
}

// The head's max |dO_q|^2 and max |V_k|^2 from the per-block maxima.  Every lane of a warp calls it.
__device__ __forceinline__ float2 max_norms(const float2* norms2, int nblk) {
  float a = 0.f, b = 0.f;
  for (int i = static_cast<int>(lane_id()); i < nblk; i += 32) {
    const float2 x = norms2[i];
    a = fmaxf(a, x.x);
    b = fmaxf(b, x.y);
  }
  for (int o = 16; o > 0; o >>= 1) {
    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, o));
  }
  return make_float2(a, b);
}

// log2 of the factor dS is multiplied by before its rounding to f16 (bf16, whose exponent range is
// fp32's, needs none): 14 - log2(2 A B) rounded down, from A^2 and B^2.  Norms of zero, or ones that are not
// finite, leave it at 0.
__device__ __forceinline__ float ds_shift(float a2, float b2) {
  // 2 A B = 2 sqrt(a2 b2); the sum of logs cannot overflow
  const float l = 1.f + 0.5f * (log2f(a2) + log2f(b2));
  return l > -100.f && l < 100.f ? floorf(14.f - l) : 0.f;
}

// Shared memory and threads of one pass.  Own tiles A, B: 128 rows x HD (K and V in dkv, Q and dO in
// dq), slabs of 64 columns, 128-byte swizzle.  Two rings hold this CTA's halves of the streamed blocks,
// in two cuts of the same size: ring A "rows", R / 2 rows x HD, the B operands of the products over HD
// (S, dP); ring B "cols", R rows x HD / 2, those of the products over the rows.
template <int HD, class Shape>
struct Layout {
  static constexpr int R = Shape::R, COLS = Shape::COLS, N = Shape::SLOTS;
  static constexpr int PARTS = R / COLS;
  static constexpr int EW_WARPS = 4 * PARTS;
  static constexpr int FIRST_EW = 3;  // after the loading and the two issuing warps
  static constexpr int THREADS = 32 * (FIRST_EW + EW_WARPS);
  static constexpr int NV = Shape::VECS, OUT = Shape::OUT;
  static constexpr int SLAB = T * 128;
  static constexpr int TILE = (HD / 64) * SLAB;
  static constexpr int RSLAB = R / 2 * 128;
  static constexpr int CUT = R * HD;
  static constexpr int SLOT_A = 2 * CUT, SLOT_B = Shape::CUTS_B * CUT;
  static constexpr int OFF_A = 0;
  static constexpr int OFF_B = OFF_A + TILE;
  static constexpr int OFF_RING_A = OFF_B + TILE;
  static constexpr int OFF_RING_B = OFF_RING_A + N * SLOT_A;
  static constexpr int OFF_VEC = OFF_RING_B + N * SLOT_B;  // dkv: [NV][nlse2 | ndelta], R each
  static constexpr int OUT_PARTS = PARTS < 4 ? PARTS : 4;  // parts that store
  static constexpr int OFF_OUT = OFF_VEC + NV * 2 * R * 4;  // [4 OUT_PARTS warps][32 rows][OUT]
  static constexpr int END = OFF_OUT + 4 * OUT_PARTS * 32 * OUT * 2;
  static constexpr int NUM_BARS = 4 * N + 4 + NV + 11;
  static_assert(RSLAB % 1024 == 0 && CUT % 1024 == 0, "swizzled tiles keep their alignment");
  static_assert(R % 16 == 0 && R % COLS == 0 && OFF_VEC % 16 == 0 && (R * 4) % 16 == 0, "bulk copies");
  static_assert(OFF_OUT % 128 == 0 && (32 * OUT * 2) % 128 == 0, "staged pieces are TMA boxes");
};

// One own tile of 128 rows x HD; its completion is counted by the leader's barrier.
template <class L, int HD>
__device__ __forceinline__ void load_tile(uint8_t* dst, const CUtensorMap* m, uint32_t bar, int x, int y, int z) {
  for (int c = 0; c < HD / 64; ++c) tma_load_3d_pair(dst + c * L::SLAB, m, bar, x + 64 * c, y, z);
}
// This CTA's half of a block in either cut.
template <class L, int HD>
__device__ __forceinline__ void load_rows_cut(uint8_t* dst, const CUtensorMap* m, uint32_t bar, int x, int y, int z,
                                              int rank) {
  for (int c = 0; c < HD / 64; ++c)
    tma_load_3d_pair(dst + c * L::RSLAB, m, bar, x + 64 * c, y + L::R / 2 * rank, z);
}
template <int HD>
__device__ __forceinline__ void load_cols_cut(uint8_t* dst, const CUtensorMap* m, uint32_t bar, int x, int y, int z,
                                              int rank) {
  tma_load_3d_pair(dst, m, bar, x + rank * (HD / 2), y, z);
}

// The descriptor of the same layout `bytes` further on.  One 32-bit add: the start address (in 16-byte
// units) fills the low 14 bits and stays below 2^14 inside 227 KB.
__device__ __forceinline__ uint64_t desc_at(uint64_t d, uint32_t bytes) {
  return (d & 0xFFFFFFFF00000000ull) | (static_cast<uint32_t>(d) + (bytes >> 4));
}

// D[256 x R] = A B^T over HD: A both CTAs' own tiles, B a block in the rows cut.
template <class L, int HD, int F>
__device__ __forceinline__ void mma_rows(uint32_t d, const uint8_t* a, const uint8_t* b) {
  constexpr uint32_t idesc = idesc_f16kind(2 * T, L::R, F == FMT_F16, false, false);
  const uint64_t ad = smem_desc_sw128(smem_u32(a), 16, 1024), bd = smem_desc_sw128(smem_u32(b), 16, 1024);
#pragma unroll
  for (int kk = 0; kk < HD / 16; ++kk)
    mma_f16kind_ss_pair(d, desc_at(ad, (kk >> 2) * L::SLAB + (kk & 3) * 32),
                        desc_at(bd, (kk >> 2) * L::RSLAB + (kk & 3) * 32), idesc, kk > 0 ? 1u : 0u);
}

// D[256 x HD] (+)= A[256 x R] B: A as 16-bit pairs in R / 2 TMEM columns, B a block in the cols cut, its
// rows being the contraction axis.
template <class L, int HD, int F>
__device__ __forceinline__ void mma_cols(uint32_t d, uint32_t a, const uint8_t* b, bool accumulate) {
  constexpr uint32_t idesc = idesc_f16kind(2 * T, HD, F == FMT_F16, false, true);
  const uint64_t bd = HD == 128 ? smem_desc_sw128(smem_u32(b), 16, 8 * HD) : smem_desc_sw64(smem_u32(b), 16, 8 * HD);
#pragma unroll
  for (int kk = 0; kk < L::R / 16; ++kk)  // 16 rows of HD / 2 values
    mma_f16kind_ts_pair(d, a + 8 * kk, desc_at(bd, kk * 16 * HD), idesc, (accumulate || kk > 0) ? 1u : 0u);
}

// COLS fp32 columns of this thread's TMEM lane.
__device__ __forceinline__ void get_cols(uint32_t taddr, uint32_t (&r)[32]) { tmem_ld32(taddr, r); }
__device__ __forceinline__ void get_cols(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// Wait for this thread's TMEM loads; no use of r can move above it.
__device__ __forceinline__ void got_cols(uint32_t (&r)[32]) { tmem_ld_wait_regs(r); }
__device__ __forceinline__ void got_cols(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
  asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
               "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
}
// COLS / 2 columns of 16-bit pairs.
__device__ __forceinline__ void put_cols(uint32_t taddr, const uint32_t (&r)[16]) { tmem_st16(taddr, r); }
__device__ __forceinline__ void put_cols(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ float2 as_f2(const uint32_t* r) {
  return make_float2(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// OUT columns of this warp's 32 accumulator rows (fp32 at taddr) times f, rounded to 16 bits, staged in
// shared memory and stored as one TMA box (x, y) of element z; rows that take no part as zeros, rows past
// the sequence are cut off by the tensor map.  Stored from registers, a row per lane, the same tiles
// took 7000 clocks a work item of 100,000.
template <int OUT, int F>
__device__ __forceinline__ void store_box(const CUtensorMap* m, uint8_t* stage, uint32_t taddr, float f, bool live,
                                          int x, int y, int z) {
  uint32_t raw[OUT];
  get_cols(taddr, raw);
  bulk_wait_group_read<0>();  // lane 0's previous box has left the buffer
  __syncwarp();
  got_cols(raw);
#pragma unroll
  for (int q = 0; q < OUT / 8; ++q) {
    float o[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) o[k] = live ? __uint_as_float(raw[8 * q + k]) * f : 0.f;
    store8<F, false>(stage + lane_id() * (2 * OUT), q, o);
  }
  fence_proxy_async_smem();
  __syncwarp();
  if (lane_id() == 0) {
    tma_store_3d(m, stage, x, y, z);
    bulk_commit_group();
  }
  __syncwarp();
}

// Zeros into this CTA's 128 rows from row0, those below seq, of one head; t: index among the N
// elementwise threads.
template <int HD, int N>
__device__ __forceinline__ void zero_rows(uint16_t* base, int64_t ld, int row0, int seq, int t) {
  constexpr int LANES = HD / 8;
  for (int i = t; i < T * LANES; i += N) {
    const int row = row0 + i / LANES;
    if (row < seq) reinterpret_cast<uint4*>(base + row * ld)[i % LANES] = make_uint4(0u, 0u, 0u, 0u);
  }
}

// A gradient: its rows (for zeros), and the map of its boxes of 32 rows.
struct OutRows {
  uint16_t* p;
  int64_t ld;
};

// A ring of N slots; u counts uses (monotonic over all work items).
template <int N>
struct Ring {
  uint64_t *full, *empty;
  __device__ __forceinline__ Ring(uint64_t* b) : full(b), empty(b + N) {}
  static __device__ __forceinline__ int slot(int u) { return u % N; }
  static __device__ __forceinline__ uint32_t phase(int u) { return static_cast<uint32_t>(u / N) & 1u; }
  __device__ __forceinline__ void init() const {
    for (int i = 0; i < N; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
  }
  __device__ __forceinline__ bool wait_full(int u, const KernelGuard& g, volatile uint32_t* abort_flag,
                                            uint32_t where) const {
    return mbar_wait(&full[slot(u)], phase(u), g, abort_flag, where);
  }
  __device__ __forceinline__ bool wait_empty(int u, const KernelGuard& g, volatile uint32_t* abort_flag,
                                             uint32_t where) const {
    return mbar_wait_warp(&empty[slot(u)], phase(u) ^ 1u, g, abort_flag, where);
  }
  // The leader arms the barrier for both CTAs' halves; returns its shared::cluster address.
  __device__ __forceinline__ uint32_t arm(int u, bool leader, uint32_t bytes) const {
    if (leader) mbar_arrive_expect_tx(&full[slot(u)], bytes);
    return mapa_shared(smem_u32(&full[slot(u)]), 0);
  }
  // Wait for the copies of the last uses (leaving with copies in flight is not allowed).
  __device__ __forceinline__ void drain(int uses, const KernelGuard& g, volatile uint32_t* abort_flag,
                                        uint32_t where) const {
    for (int u = uses > N ? uses - N : 0; u < uses; ++u) mbar_wait(&full[slot(u)], phase(u), g, abort_flag, where, true);
  }
};

// Work item of a CTA pair: 256 rows (tile tt) of one head of one element.
struct Item {
  int b, head, tt, n, nb;  // n: tokens of the element; nb: blocks of the other axis (0: no row takes part)
  int64_t bh;
};
// The items in the order in which the pairs are dealt them, pair p taking p, p + pairs, ...  In a padded
// batch the tiles that hold tokens come first, element by element, then the others, which are only zeroed:
// with every element's tiles together the pairs' shares of the products came out uneven (1535, 1100, 1324
// and 1023 tokens padded to 1535, 16 heads of 64: 148 us against 139; 128 channels: 187 against 173).  Elements
// of one tile stay together: they are uneven by a few blocks at most, and finding the place costs more
// (512 elements of 80 or 10 tokens x 4 heads of 64: 191 us, in the other order 210).
// Items are asked for in rising order, by whole warps: lane l holds the tiles of element chunk + l, summed
// over the lanes up to it.
template <int R>
struct Items {
  int batch, ntile, n_heads, seq;
  const int32_t* key_lens;
  int total, live;  // items; the first `live` hold tokens (elements of one tile: unless they have none)
  int chunk = 0, base = 0, upto = 0;
  bool past = false;

  __device__ Items(int batch, int n_heads, int seq, const int32_t* key_lens)
      : batch(batch), ntile((seq + 2 * T - 1) / (2 * T)), n_heads(n_heads), seq(seq), key_lens(key_lens) {
    total = live = batch * n_heads * ntile;
    if (key_lens == nullptr || ntile == 1) return;
    int tiles = 0;
    for (int e = static_cast<int>(lane_id()); e < batch; e += 32) tiles += tiles_of(e);
    live = n_heads * __reduce_add_sync(0xffffffffu, tiles);
    sum_chunk();
  }
  __device__ __forceinline__ int tiles_of(int e) const { return (tokens_of(key_lens, e, seq) + 2 * T - 1) / (2 * T); }
  __device__ __forceinline__ void sum_chunk() {
    const int lane = static_cast<int>(lane_id()), e = chunk + lane;
    upto = e >= batch ? 0 : past ? ntile - tiles_of(e) : tiles_of(e);
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
  }
  __device__ __forceinline__ Item at(int i) {
    Item it;
    if (key_lens == nullptr || ntile == 1) {
      it.tt = i % ntile;
      const int bh = i / ntile;
      it.head = bh % n_heads;
      it.b = bh / n_heads;
      it.n = tokens_of(key_lens, it.b, seq);
    } else {
      if (i >= live && !past) {
        past = true;
        chunk = 0;
        base = live;
        sum_chunk();
      }
      while (chunk + 32 < batch) {
        const int all = n_heads * __shfl_sync(0xffffffffu, upto, 31);
        if (i - base < all) break;
        base += all;
        chunk += 32;
        sum_chunk();
      }
      const int k = min(__popc(__ballot_sync(0xffffffffu, i - base >= n_heads * upto)), 31);
      const int before = __shfl_sync(0xffffffffu, upto, max(k - 1, 0)) * (k > 0);
      const int w = max(__shfl_sync(0xffffffffu, upto, k) - before, 1), r = i - base - n_heads * before;
      it.b = chunk + k;
      it.n = tokens_of(key_lens, it.b, seq);
      it.head = r / w;
      it.tt = r % w + (past ? tiles_of(it.b) : 0);
    }
    it.bh = static_cast<int64_t>(it.b) * n_heads + it.head;
    it.nb = past ? 0 : (it.n + R - 1) / R;  // 0 too for an element of no tokens
    return it;
  }
};

// What both passes share: two CTAs on two SMs (a cluster) own 256 rows of one head, 128 each, and walk
// the other axis in blocks; the pair MMA (cta_group::2, M = 256) lets each CTA hold half of every block.
// The kernel is persistent (pair p takes items first, first + pairs, ...; rings and barrier phases run on
// across a pass's items) and every buffer between two steps has a barrier for each direction, so that a step
// waits for its own operands only and nothing relies on the order of issue:
//   warp 0            loads: the item's own tiles, per block ring A, ring B (and dkv's row vectors)
//   warp 1, leader    S(u) once S(u-1) has been read into registers, dP(u) likewise
//   warp 2, leader    the products with P and dS, once those are written (warp 2 holds the TMEM)
//   the others        the elementwise step; thread = own row and COLS columns of the block
// A wait gives up after a limit.  Its warp then goes on to the end of the block (on whatever it finds; the
// error word is set) and leaves by a vote of its lanes: leaving lane by lane could split the warp, and a vote
// at every wait cost 3 %.  Only the loads ask at once, since they may not arm a barrier that is in use; for the same
// reason an issuing lane whose wait gave up issues and commits nothing more, so that no slot counts as free before its
// copies have landed.
// One lane of each issuing warp per pair runs the tensor cores of both SMs; with one warp for all
// products its waits and commits took 1500 clocks a block, as long as the products.
template <class L, int HD>
struct Pipe {
  uint8_t *tile_a, *tile_b, *mem_a, *mem_b;
  float* vec;
  Ring<1> at, bt;
  Ring<L::N> ra, rb;
  uint64_t *vec_full, *s_full, *s_empty, *dp_full, *dp_empty, *p_full, *p_empty, *ds_full, *ds_empty, *acc_full, *acc_empty,
      *drain_bar;
  uint32_t* tmem_slot;
  volatile uint32_t* abort_flag;

  __device__ __forceinline__ Pipe(uint8_t* smem, uint64_t* bars, uint8_t* misc)
      : tile_a(smem + L::OFF_A),
        tile_b(smem + L::OFF_B),
        mem_a(smem + L::OFF_RING_A),
        mem_b(smem + L::OFF_RING_B),
        vec(reinterpret_cast<float*>(smem + L::OFF_VEC)),
        at(bars),
        bt(bars + 2),
        ra(bars + 4),
        rb(bars + 4 + 2 * L::N) {
    vec_full = bars + 4 + 4 * L::N;  // [NV] this CTA's copies
    s_full = vec_full + L::NV;
    s_empty = s_full + 1;      // leader; by every elementwise warp of both CTAs, as the ones marked *
    dp_full = s_empty + 1;
    dp_empty = dp_full + 1;    // *
    p_full = dp_empty + 1;     // *
    p_empty = p_full + 1;
    ds_full = p_empty + 1;     // *
    ds_empty = ds_full + 1;
    acc_full = ds_empty + 1;
    acc_empty = acc_full + 1;  // *
    drain_bar = acc_empty + 1;
    tmem_slot = reinterpret_cast<uint32_t*>(misc);
    abort_flag = reinterpret_cast<volatile uint32_t*>(misc + 4);
  }
  __device__ __forceinline__ void init() const {
    at.init();
    bt.init();
    ra.init();
    rb.init();
    for (int i = 0; i < L::NV; ++i) mbar_init(&vec_full[i], 1);
    for (uint64_t* b : {s_full, dp_full, p_empty, ds_empty, acc_full}) mbar_init(b, 1);
    for (uint64_t* b : {s_empty, dp_empty, p_full, ds_full, acc_empty}) mbar_init(b, 2 * L::EW_WARPS);
    mbar_init(drain_bar, 2);  // both issuing warps
    *abort_flag = 0u;
    fence_barrier_init();
  }
};

// Warp 1 of the leader: S and dP of every block.
template <class L, int HD, int F>
__device__ __forceinline__ void issue_s_dp(const Pipe<L, HD>& p, uint32_t t_s, uint32_t t_dp, int first, int pairs,
                                           Items<L::R>& items, const KernelGuard& guard) {
  const bool one = elect_one();
  auto where = [&](int k, int i) { return where_code(ERR_TIMEOUT_ABWD_MMA, k, i); };
  bool ok = true;
  int u = 0, ui = 0;
  for (int i = first; i < items.live && ok; i += pairs) {
    const int nb = items.at(i).nb;
    if (nb == 0) continue;
    ok = __all_sync(0xffffffffu, p.at.wait_full(ui, guard, p.abort_flag, where(0, u)));
    for (int j = 0; j < nb && ok; ++j, ++u) {
      const uint32_t prev = static_cast<uint32_t>(u - 1) & 1u;
      const uint8_t* slot = p.mem_a + (u % L::N) * L::SLOT_A;
      ok &= p.ra.wait_full(u, guard, p.abort_flag, where(1, u));
      ok &= u == 0 || mbar_wait(p.s_empty, prev, guard, p.abort_flag, where(2, u));
      tc_fence_after();
      if (one && ok) {
        mma_rows<L, HD, F>(t_s, p.tile_a, slot);
        mma_commit_pair(p.s_full, 0x3);
        if (j + 1 == nb) mma_commit_pair(&p.at.empty[0], 0x3);
      }
      __syncwarp();
      ok &= j > 0 || p.bt.wait_full(ui, guard, p.abort_flag, where(3, u));
      ok &= u == 0 || mbar_wait(p.dp_empty, prev, guard, p.abort_flag, where(4, u));
      tc_fence_after();
      if (one && ok) {
        mma_rows<L, HD, F>(t_dp, p.tile_b, slot + L::CUT);
        mma_commit_pair(p.dp_full, 0x3);
        mma_commit_pair(&p.ra.empty[u % L::N], 0x3);
        if (j + 1 == nb) mma_commit_pair(&p.bt.empty[0], 0x3);
      }
      ok = __all_sync(0xffffffffu, ok);
    }
    ++ui;
  }
  if (one) mma_commit_pair(p.drain_bar, 0x3);
  __syncwarp();
}

// Copies a CTA may still have in flight when it leaves: the leader's barriers count both CTAs', and the
// peer is held by the final cluster barrier until the leader has drained.
template <class L, int HD>
__device__ __forceinline__ void drain_loads(const Pipe<L, HD>& p, int n_at, int n_bt, int n_a, int n_b, int n_vec,
                                            int rank, const KernelGuard& guard) {
  const uint32_t wd = where_code(ERR_TIMEOUT_ABWD_DRAIN, rank, 0);
  if constexpr (L::NV > 0) {
    for (int v = n_vec > L::NV ? n_vec - L::NV : 0; v < n_vec; ++v)
      mbar_wait(&p.vec_full[v % L::NV], static_cast<uint32_t>(v / L::NV) & 1u, guard, p.abort_flag, wd, true);
  }
  if (rank == 0) {
    p.at.drain(n_at, guard, p.abort_flag, wd);
    p.bt.drain(n_bt, guard, p.abort_flag, wd);
    p.ra.drain(n_a, guard, p.abort_flag, wd);
    p.rb.drain(n_b, guard, p.abort_flag, wd);
  }
}

struct BwdArgs {
  const float *nlse2, *ndelta, *rows2;
  const float2* norms2;
  OutRows dq, dk, dv;
  const int32_t* key_lens;
  int batch, seq, n_heads;
};

// ------------------------------------------------------------------ dK, dV

// Own rows: keys; streamed: queries.  The products run with the keys as rows (S^T = K Q^T,
// dP^T = V dO^T), so that P^T and dS^T come out of the elementwise step in the layout in which the tensor
// core reads an A operand from TMEM: dV += P^T dO, dK += dS^T Q.
// Blocks of 80 queries at head dim 128: S^T 80, dP^T 80, P^T 40 and dS^T 40 columns beside dV and dK (128 each) are what
// TMEM holds with a region of its own for each.  With 128 and P^T over S^T, dS^T over dP^T, S(j+1) waited for
// dV(j) and dP(j+1) for dK(j): 3420 clocks a block against the products' 2048; with 96 and only
// dS^T over dP^T 2030 against 1536.
// As a launch of its own, 4608 queries and keys x 32 heads of 128 in f16: 517 us for the four products (1350
// TFLOP/s; a large library product holds 1408 in a long run) at the 1.51 GHz that the power limit leaves, the
// tensor core busy in 74 % of the cycles.  Bound by that limit and by the hand-over of S, P, dP and dS between
// the tensor core and the elementwise warps.  64 heads of 64 in bf16: 658 us (1060 TFLOP/s).
struct DkvMaps {
  CUtensorMap k, v, q_rows, q_cols, do_rows, do_cols, tq_rows, tq_cols, tdo_rows, tdo_cols, dk, dv;
};
template <int HD>
using DkvLayout = Layout<HD, DkvShape<HD>>;

template <int HD, int F>
__device__ __forceinline__ void dkv_pass(const Pipe<DkvLayout<HD>, HD>& p, uint8_t* smem, uint32_t tmem,
                                         const DkvMaps& tm, const BwdArgs& a, const KernelGuard& guard) {
  using L = DkvLayout<HD>;
  constexpr int R = L::R, COLS = L::COLS, N = L::N, NV = L::NV;
  const float *nlse2 = a.nlse2, *ndelta = a.ndelta;
  const float2* norms2 = a.norms2;
  const OutRows dk = a.dk, dv = a.dv;
  const int seq = a.seq;
  const int warp = static_cast<int>(warp_id());
  const int lane = static_cast<int>(lane_id());
  const int rank = static_cast<int>(cluster_ctarank());
  const bool leader = rank == 0;
  const int first = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int nblk = blocks_of(seq) + 1;
  Items<R> items(a.batch, a.n_heads, seq, a.key_lens);
  constexpr int C_DP = R, C_P = 2 * R, C_DS = C_P + R / 2, C_DV = TMEM_COLS - 2 * HD, C_DK = TMEM_COLS - HD;
  static_assert(C_DS + R / 2 <= C_DV, "TMEM columns");

  if (warp == 0) {
    const bool one = elect_one();
    int u = 0, ui = 0, n_b = 0, n_bt = 0, n_at = 0;
    bool ok = true;
    auto where = [&](int i) { return where_code(ERR_TIMEOUT_ABWD_PRODUCER, rank, i); };
    for (int i = first; i < items.live && ok; i += pairs) {
      const Item it = items.at(i);
      if (it.nb == 0) continue;
      const bool tail = has_tail(it.n, seq, R);
      const int x = it.head * HD, row0 = it.tt * 2 * T + rank * T;
      ok = p.at.wait_empty(ui, guard, p.abort_flag, where(0xFFFF));
      if (!ok) break;
      if (one) load_tile<L, HD>(p.tile_a, &tm.k, p.at.arm(ui, leader, 2 * L::TILE), x, row0, it.b);
      ++n_at;
      __syncwarp();
      for (int j = 0; j < it.nb && ok; ++j) {
        const bool tl = tail && j == it.nb - 1;
        const int y = tl ? 0 : j * R, sv = u % NV;
        // the slot is free when dP(u - N) is done; that product waited until every warp was done with dP of
        // the block before, so with all blocks up to u - 5, whose row vectors' slot is reused here
        ok = p.ra.wait_empty(u, guard, p.abort_flag, where(u));
        if (!ok) break;
        if (one) {
          uint8_t* slot = p.mem_a + (u % N) * L::SLOT_A;
          const uint32_t bar = p.ra.arm(u, leader, 2 * L::SLOT_A);
          load_rows_cut<L, HD>(slot, tl ? &tm.tq_rows : &tm.q_rows, bar, x, y, it.b, rank);
          load_rows_cut<L, HD>(slot + L::CUT, tl ? &tm.tdo_rows : &tm.do_rows, bar, x, y, it.b, rank);
          float* vec = p.vec + sv * 2 * R;
          mbar_arrive_expect_tx(&p.vec_full[sv], 2 * R * 4);
          bulk_load(vec, nlse2 + it.bh * nblk * T + j * R, R * 4, &p.vec_full[sv]);
          bulk_load(vec + R, ndelta + it.bh * nblk * T + j * R, R * 4, &p.vec_full[sv]);
        }
        __syncwarp();
        ++u;
        if (j == 0) {
          ok = p.bt.wait_empty(ui, guard, p.abort_flag, where(0xFFFE));
          if (!ok) break;
          if (one) load_tile<L, HD>(p.tile_b, &tm.v, p.bt.arm(ui, leader, 2 * L::TILE), x, row0, it.b);
          ++n_bt;
          __syncwarp();
        }
        ok = p.rb.wait_empty(n_b, guard, p.abort_flag, where(n_b));
        if (!ok) break;
        if (one) {
          uint8_t* slot = p.mem_b + (n_b % N) * L::SLOT_B;
          const uint32_t bar = p.rb.arm(n_b, leader, 2 * L::SLOT_B);
          load_cols_cut<HD>(slot, tl ? &tm.tdo_cols : &tm.do_cols, bar, x, y, it.b, rank);
          load_cols_cut<HD>(slot + L::CUT, tl ? &tm.tq_cols : &tm.q_cols, bar, x, y, it.b, rank);
        }
        ++n_b;
        __syncwarp();
      }
      ++ui;
    }
    drain_loads(p, n_at, n_bt, u, n_b, u, rank, guard);
  } else if (warp == 1) {
    if (leader)
      issue_s_dp<L, HD, F>(p, tmem, tmem + C_DP, first, pairs, items, guard);
    mbar_wait(p.drain_bar, 0u, guard, p.abort_flag, where_code(ERR_TIMEOUT_ABWD_DRAIN, rank, 1), true);
  } else if (warp == 2) {
    if (leader) {
      const bool one = elect_one();
      auto where = [&](int k, int i) { return where_code(ERR_TIMEOUT_ABWD_MMA, k, i); };
      bool ok = true;
      int u = 0, ui = 0;
      for (int i = first; i < items.live && ok; i += pairs) {
        const int nb = items.at(i).nb;
        if (nb == 0) continue;
        // the first dV of an item overwrites accumulators that both CTAs must have read
        ok = ui == 0 || mbar_wait_warp(p.acc_empty, static_cast<uint32_t>(ui - 1) & 1u, guard, p.abort_flag, where(5, u));
        for (int j = 0; j < nb && ok; ++j, ++u) {
          const uint32_t par = static_cast<uint32_t>(u) & 1u;
          const uint8_t* slot = p.mem_b + (u % N) * L::SLOT_B;
          ok &= p.rb.wait_full(u, guard, p.abort_flag, where(6, u));
          ok &= mbar_wait(p.p_full, par, guard, p.abort_flag, where(7, u));
          tc_fence_after();
          if (one && ok) {
            mma_cols<L, HD, F>(tmem + C_DV, tmem + C_P, slot, j > 0);
            mma_commit_pair(p.p_empty, 0x3);
          }
          __syncwarp();
          ok &= mbar_wait(p.ds_full, par, guard, p.abort_flag, where(8, u));
          tc_fence_after();
          if (one && ok) {
            mma_cols<L, HD, F>(tmem + C_DK, tmem + C_DS, slot + L::CUT, j > 0);
            mma_commit_pair(p.ds_empty, 0x3);
            mma_commit_pair(&p.rb.empty[u % N], 0x3);
          }
          ok = __all_sync(0xffffffffu, ok);
        }
        if (ok && one) mma_commit_pair(p.acc_full, 0x3);
        __syncwarp();
        ++ui;
      }
      if (one) mma_commit_pair(p.drain_bar, 0x3);
      __syncwarp();
    }
    mbar_wait(p.drain_bar, 0u, guard, p.abort_flag, where_code(ERR_TIMEOUT_ABWD_DRAIN, rank, 2), true);
  } else if (warp < L::FIRST_EW + L::EW_WARPS) {
    const int part = (warp - L::FIRST_EW) >> 2;
    const int quarter = warp & 3;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t s_col = lanes + COLS * part, dp_col = s_col + C_DP;
    const uint32_t p_col = lanes + C_P + COLS / 2 * part, ds_col = lanes + C_DS + COLS / 2 * part;
    const float scale = HD == 128 ? 0.08838834764831845f : 0.125f;
    const float2 c2 = make_float2(scale * LOG2E, scale * LOG2E);
    auto where = [&](int k, int i) { return where_code(ERR_TIMEOUT_ABWD_SOFTMAX, k, i); };
    bool ok = true;
    // (a copy of row vectors may be on its way into a slot whose wait gave up: no arrive then)
    auto arrive = [&](uint64_t* bar) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0 && ok) mbar_arrive_remote(mapa_shared(smem_u32(bar), 0));
    };
    uint8_t* stage = smem + L::OFF_OUT + (warp - L::FIRST_EW) * 32 * L::OUT * 2;
    auto shift_of = [&](int i) {
      if (F != FMT_F16 || i >= items.live) return 0.f;
      const Item it = items.at(i);
      const float2 m = max_norms(norms2 + it.bh * nblk, blocks_of(it.n));
      return ds_shift(m.x, m.y);
    };
    int u = 0, ui = 0;
    float shift = shift_of(first);
    for (int i = first; i < items.total && ok; i += pairs) {
      const Item it = items.at(i);
      const int row0 = it.tt * 2 * T + rank * T;
      if (it.nb == 0) {
        shift = shift_of(i + pairs);
        const int t = static_cast<int>(threadIdx.x) - 32 * L::FIRST_EW;
        zero_rows<HD, 32 * L::EW_WARPS>(dk.p + static_cast<int64_t>(it.b) * seq * dk.ld + it.head * HD, dk.ld, row0, seq, t);
        zero_rows<HD, 32 * L::EW_WARPS>(dv.p + static_cast<int64_t>(it.b) * seq * dv.ld + it.head * HD, dv.ld, row0, seq, t);
        continue;
      }
      // P carries 2^15 in f16; dS = that P times (dP - delta) times tau = 2^(shift - 15)
      const float tau = F == FMT_F16 ? exp2f(shift - P_SHIFT) : 1.f;
      for (int j = 0; j < it.nb && ok; ++j, ++u) {
        const uint32_t par = static_cast<uint32_t>(u) & 1u;
        const int sv = u % NV;
        const float* vec = p.vec + sv * 2 * R + COLS * part;
        ok &= mbar_wait(&p.vec_full[sv], static_cast<uint32_t>(u / NV) & 1u, guard, p.abort_flag, where(0, u));
        ok &= mbar_wait(p.s_full, par, guard, p.abort_flag, where(1, u));
        tc_fence_after();
        uint32_t raw[COLS];
        get_cols(s_col, raw);
        got_cols(raw);
        arrive(p.s_empty);
        float e[COLS];
        uint32_t pk[COLS / 2];
#pragma unroll
        for (int k = 0; k < COLS; k += 2) {
          const float2 x = fma2(as_f2(raw + k), c2, *reinterpret_cast<const float2*>(vec + k));
          e[k] = ex2_approx(x.x);
          e[k + 1] = ex2_approx(x.y);
          pk[k / 2] = pack2<F, false>(e[k], e[k + 1]);
        }
        ok &= mbar_wait(p.p_empty, par ^ 1u, guard, p.abort_flag, where(2, u));  // dV(u - 1) has read P
        tc_fence_after();
        put_cols(p_col, pk);
        tmem_st_wait();
        arrive(p.p_full);
        ok &= mbar_wait(p.dp_full, par, guard, p.abort_flag, where(3, u));
        tc_fence_after();
        get_cols(dp_col, raw);
        got_cols(raw);
        arrive(p.dp_empty);
#pragma unroll
        for (int k = 0; k < COLS; k += 2) {
          float2 y = mul2(add2(as_f2(raw + k), *reinterpret_cast<const float2*>(vec + R + k)),
                          make_float2(e[k], e[k + 1]));
          if constexpr (F == FMT_F16) y = mul2(y, make_float2(tau, tau));
          pk[k / 2] = pack2<F, false>(y.x, y.y);
        }
        ok &= mbar_wait(p.ds_empty, par ^ 1u, guard, p.abort_flag, where(4, u));  // dK(u - 1) has read dS
        tc_fence_after();
        put_cols(ds_col, pk);
        tmem_st_wait();
        arrive(p.ds_full);
        ok = __all_sync(0xffffffffu, ok);
      }
      if (!ok) break;
      const float fv = F == FMT_F16 ? exp2f(-P_SHIFT) : 1.f, fk = scale * exp2f(-shift);
      shift = shift_of(i + pairs);  // the next item's, while the last products run
      ok = mbar_wait_warp(p.acc_full, static_cast<uint32_t>(ui) & 1u, guard, p.abort_flag, where(5, u));
      if (!ok) break;
      tc_fence_after();
      // 2 HD / OUT pieces of the rows (dV's, then dK's), dealt to the rows' warps in turn
      const int row = row0 + 32 * quarter;
      for (int c = part; part < L::OUT_PARTS && c < 2 * HD / L::OUT; c += L::OUT_PARTS) {
        const bool is_v = c < HD / L::OUT;
        const int col = L::OUT * (is_v ? c : c - HD / L::OUT);
        store_box<L::OUT, F>(is_v ? &tm.dv : &tm.dk, stage, lanes + (is_v ? C_DV : C_DK) + col, is_v ? fv : fk,
                             row + lane < it.n, it.head * HD + col, row, it.b);
      }
      arrive(p.acc_empty);
      ++ui;
    }
    bulk_wait_group<0>();  // the last boxes are in memory
  }
}

// ------------------------------------------------------------------ dQ

// Own rows: queries; streamed: keys in blocks of 128.  S = Q K^T and dP = dO V^T, dS = P (dP - delta) as an
// A operand in TMEM, dQ += dS K.  TMEM: S | dP | dS (64 columns) | dQ.  lse and delta are per thread.
// As a launch of its own with 95 registers a thread, 4608 x 32 heads of 128 in f16: 372 us for three products
// (1400 TFLOP/s) at 1.52 GHz, the tensor core busy in 76 % of the cycles, the exponentials' unit in 57 %.  Bound as
// the key pass.  64 heads of 64: 505 us.
struct DqMaps {
  CUtensorMap q, dout, k_rows, k_cols, v_rows, tk_rows, tk_cols, dq;
};
template <int HD>
using DqLayout = Layout<HD, DqShape>;

template <int HD, int F>
__device__ __forceinline__ void dq_pass(const Pipe<DqLayout<HD>, HD>& p, uint8_t* smem, uint32_t tmem,
                                        const DqMaps& tm, const BwdArgs& a, const KernelGuard& guard) {
  using L = DqLayout<HD>;
  constexpr int R = L::R, COLS = L::COLS, N = L::N;
  // columns of dP in registers at a time: at head dim 128 the key pass's threads leave 80 registers each, and
  // two steps cost 861 us where one, spilling, cost 883 (4608 tokens x 32 heads, bf16)
  constexpr int STEP = HD == 128 ? 16 : COLS;
  const float *nlse2 = a.nlse2, *ndelta = a.ndelta;
  const OutRows dq = a.dq;
  const int seq = a.seq;
  const int warp = static_cast<int>(warp_id());
  const int lane = static_cast<int>(lane_id());
  const int rank = static_cast<int>(cluster_ctarank());
  const bool leader = rank == 0;
  const int pairs = gridDim.x >> 1;
  const int nblk = blocks_of(seq) + 1;
  Items<R> items(a.batch, a.n_heads, seq, a.key_lens);
  // the dealing goes on where the key pass's items that hold tokens ended
  const int first = (static_cast<int>(blockIdx.x >> 1) + pairs - items.live % pairs) % pairs;
  constexpr int C_DP = R, C_DS = 2 * R, C_DQ = 384;
  static_assert(C_DS + R / 2 <= C_DQ, "TMEM columns");

  if (warp == 0) {
    const bool one = elect_one();
    int u = 0, ui = 0, n_b = 0, n_at = 0, n_bt = 0;
    bool ok = true;
    auto where = [&](int i) { return where_code(ERR_TIMEOUT_ABWD_PRODUCER, 2 + rank, i); };
    for (int i = first; i < items.live && ok; i += pairs) {
      const Item it = items.at(i);
      if (it.nb == 0) continue;
      const bool tail = has_tail(it.n, seq, R);
      const int x = it.head * HD, row0 = it.tt * 2 * T + rank * T;
      ok = p.at.wait_empty(ui, guard, p.abort_flag, where(0xFFFF));
      if (!ok) break;
      if (one) load_tile<L, HD>(p.tile_a, &tm.q, p.at.arm(ui, leader, 2 * L::TILE), x, row0, it.b);
      ++n_at;
      __syncwarp();
      for (int j = 0; j < it.nb && ok; ++j) {
        const bool tl = tail && j == it.nb - 1;
        const int y = tl ? 0 : j * R;
        ok = p.ra.wait_empty(u, guard, p.abort_flag, where(u));
        if (!ok) break;
        if (one) {
          uint8_t* slot = p.mem_a + (u % N) * L::SLOT_A;
          const uint32_t bar = p.ra.arm(u, leader, 2 * L::SLOT_A);
          load_rows_cut<L, HD>(slot, tl ? &tm.tk_rows : &tm.k_rows, bar, x, y, it.b, rank);
          load_rows_cut<L, HD>(slot + L::CUT, &tm.v_rows, bar, x, j * R, it.b, rank);
        }
        __syncwarp();
        ++u;
        if (j == 0) {
          ok = p.bt.wait_empty(ui, guard, p.abort_flag, where(0xFFFE));
          if (!ok) break;
          if (one) load_tile<L, HD>(p.tile_b, &tm.dout, p.bt.arm(ui, leader, 2 * L::TILE), x, row0, it.b);
          ++n_bt;
          __syncwarp();
        }
        ok = p.rb.wait_empty(n_b, guard, p.abort_flag, where(n_b));
        if (!ok) break;
        if (one)
          load_cols_cut<HD>(p.mem_b + (n_b % N) * L::SLOT_B, tl ? &tm.tk_cols : &tm.k_cols,
                            p.rb.arm(n_b, leader, 2 * L::SLOT_B), x, y, it.b, rank);
        ++n_b;
        __syncwarp();
      }
      ++ui;
    }
    drain_loads(p, n_at, n_bt, u, n_b, 0, rank, guard);
  } else if (warp == 1) {
    if (leader)
      issue_s_dp<L, HD, F>(p, tmem, tmem + C_DP, first, pairs, items, guard);
    mbar_wait(p.drain_bar, 0u, guard, p.abort_flag, where_code(ERR_TIMEOUT_ABWD_DRAIN, rank, 3), true);
  } else if (warp == 2) {
    if (leader) {
      const bool one = elect_one();
      auto where = [&](int k, int i) { return where_code(ERR_TIMEOUT_ABWD_MMA, k, i); };
      bool ok = true;
      int u = 0, ui = 0;
      for (int i = first; i < items.live && ok; i += pairs) {
        const int nb = items.at(i).nb;
        if (nb == 0) continue;
        // the first dQ of an item overwrites an accumulator that both CTAs must have read
        ok = ui == 0 || mbar_wait_warp(p.acc_empty, static_cast<uint32_t>(ui - 1) & 1u, guard, p.abort_flag, where(9, u));
        for (int j = 0; j < nb && ok; ++j, ++u) {
          ok &= p.rb.wait_full(u, guard, p.abort_flag, where(10, u));
          ok &= mbar_wait(p.ds_full, static_cast<uint32_t>(u) & 1u, guard, p.abort_flag, where(11, u));
          tc_fence_after();
          if (one && ok) {
            mma_cols<L, HD, F>(tmem + C_DQ, tmem + C_DS, p.mem_b + (u % N) * L::SLOT_B, j > 0);
            mma_commit_pair(p.ds_empty, 0x3);
            mma_commit_pair(&p.rb.empty[u % N], 0x3);
          }
          ok = __all_sync(0xffffffffu, ok);
        }
        if (ok && one) mma_commit_pair(p.acc_full, 0x3);
        __syncwarp();
        ++ui;
      }
      if (one) mma_commit_pair(p.drain_bar, 0x3);
      __syncwarp();
    }
    mbar_wait(p.drain_bar, 0u, guard, p.abort_flag, where_code(ERR_TIMEOUT_ABWD_DRAIN, rank, 4), true);
  } else if (warp < L::FIRST_EW + L::EW_WARPS) {
    const int part = (warp - L::FIRST_EW) >> 2;
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t s_col = lanes + COLS * part, dp_col = s_col + C_DP, ds_col = lanes + C_DS + COLS / 2 * part;
    const float scale = HD == 128 ? 0.08838834764831845f : 0.125f;
    const float2 c2 = make_float2(scale * LOG2E, scale * LOG2E);
    auto where = [&](int k, int i) { return where_code(ERR_TIMEOUT_ABWD_SOFTMAX, k, i); };
    auto arrive = [&](uint64_t* bar) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(mapa_shared(smem_u32(bar), 0));
    };
    uint8_t* stage = smem + L::OFF_OUT + (warp - L::FIRST_EW) * 32 * L::OUT * 2;
    struct RowState {
      float nl, nd, shift;
    };
    // the padded row vectors reach past the pair's 256 rows
    auto state_of = [&](int i) {
      RowState s{0.f, 0.f, 0.f};
      if (i >= items.live) return s;
      const Item it = items.at(i);
      const int64_t at = it.bh * nblk * T + it.tt * 2 * T + rank * T + r;
      s.nl = nlse2[at];
      s.nd = ndelta[at];
      if constexpr (F == FMT_F16) s.shift = ds_shift(a.rows2[at], max_norms(a.norms2 + it.bh * nblk, blocks_of(it.n)).y);
      return s;
    };
    bool ok = true;
    int u = 0, ui = 0;
    RowState next = state_of(first);
    for (int i = first; i < items.total && ok; i += pairs) {
      const Item it = items.at(i);
      const int row0 = it.tt * 2 * T + rank * T;
      if (it.nb == 0) {
        next = state_of(i + pairs);
        zero_rows<HD, 32 * L::EW_WARPS>(dq.p + static_cast<int64_t>(it.b) * seq * dq.ld + it.head * HD, dq.ld, row0, seq,
                                        static_cast<int>(threadIdx.x) - 32 * L::FIRST_EW);
        continue;
      }
      const float nl = next.nl, nd = next.nd, shift = next.shift;
      const float tau = F == FMT_F16 ? exp2f(shift - P_SHIFT) : 1.f;
      const float2 nl2 = make_float2(nl, nl);
      // tau (dP - delta): one fma on the pair
      const float2 tau2 = make_float2(tau, tau), nd2 = make_float2(nd * tau, nd * tau);
      for (int j = 0; j < it.nb && ok; ++j, ++u) {
        const uint32_t par = static_cast<uint32_t>(u) & 1u;
        ok &= mbar_wait(p.s_full, par, guard, p.abort_flag, where(6, u));
        tc_fence_after();
        uint32_t raw[COLS];
        get_cols(s_col, raw);
        got_cols(raw);
        arrive(p.s_empty);
        float e[COLS];
#pragma unroll
        for (int k = 0; k < COLS; k += 2) {
          const float2 x = fma2(as_f2(raw + k), c2, nl2);
          e[k] = ex2_approx(x.x);
          e[k + 1] = ex2_approx(x.y);
        }
        ok &= mbar_wait(p.dp_full, par, guard, p.abort_flag, where(7, u));
        tc_fence_after();
        const int valid = it.n - j * R - COLS * part;  // keys past the tokens: dS = 0 whatever S and dP hold
        uint32_t pk[COLS / 2];
#pragma unroll
        for (int c = 0; c < COLS; c += STEP) {
          uint32_t dp[STEP];
          get_cols(dp_col + c, dp);
          got_cols(dp);
          if (c + STEP == COLS) arrive(p.dp_empty);
          if (valid < COLS) {
#pragma unroll
            for (int k = 0; k < STEP; ++k) {
              e[c + k] = c + k < valid ? e[c + k] : 0.f;
              dp[k] = c + k < valid ? dp[k] : 0u;
            }
          }
#pragma unroll
          for (int k = 0; k < STEP; k += 2) {
            const float2 v = as_f2(dp + k);
            const float2 y = mul2(F == FMT_F16 ? fma2(v, tau2, nd2) : add2(v, nd2), make_float2(e[c + k], e[c + k + 1]));
            pk[(c + k) / 2] = pack2<F, false>(y.x, y.y);
          }
        }
        ok &= mbar_wait(p.ds_empty, par ^ 1u, guard, p.abort_flag, where(8, u));  // dQ(u - 1) has read dS
        tc_fence_after();
        put_cols(ds_col, pk);
        tmem_st_wait();
        arrive(p.ds_full);
        ok = __all_sync(0xffffffffu, ok);
      }
      if (!ok) break;
      next = state_of(i + pairs);  // while the last products run
      ok = mbar_wait_warp(p.acc_full, static_cast<uint32_t>(ui) & 1u, guard, p.abort_flag, where(9, u));
      if (!ok) break;
      tc_fence_after();
      const float fq = scale * exp2f(-shift);
      const int row = row0 + 32 * quarter;
      for (int c = part; part < L::OUT_PARTS && c < HD / L::OUT; c += L::OUT_PARTS)
        store_box<L::OUT, F>(&tm.dq, stage, lanes + C_DQ + L::OUT * c, fq, row + lane < it.n, it.head * HD + L::OUT * c,
                             row, it.b);
      arrive(p.acc_empty);
      ++ui;
    }
    bulk_wait_group<0>();  // the last boxes are in memory
  }
}

// ------------------------------------------------------------------ both passes

struct BwdMaps {
  DkvMaps dkv;
  DqMaps dq;
};

// Shared memory of the kernel: the passes' buffers in the same place, then each pass's own barriers (so that
// none is set up twice).
template <int HD>
struct Shared {
  using K = DkvLayout<HD>;
  using Q = DqLayout<HD>;
  static constexpr int THREADS = K::THREADS > Q::THREADS ? K::THREADS : Q::THREADS;
  static constexpr int OFF_BAR_K = K::END > Q::END ? K::END : Q::END;
  static constexpr int OFF_BAR_Q = OFF_BAR_K + K::NUM_BARS * 8;
  static constexpr int OFF_MISC = OFF_BAR_Q + Q::NUM_BARS * 8;
  static constexpr int SMEM = OFF_MISC + 16 + 1024;
  static_assert(SMEM <= 232448, "227 KB of shared memory per CTA");
  static __device__ __forceinline__ uint8_t* base() {
    extern __shared__ uint8_t smem_raw[];
    return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  }
  static __device__ __forceinline__ Pipe<K, HD> keys() {
    return {base(), reinterpret_cast<uint64_t*>(base() + OFF_BAR_K), base() + OFF_MISC};
  }
  static __device__ __forceinline__ Pipe<Q, HD> queries() {
    return {base(), reinterpret_cast<uint64_t*>(base() + OFF_BAR_Q), base() + OFF_MISC};
  }
};

// The passes as calls: inlined one after the other the second came out up to 25 % slower.  What they need of the
// arguments comes by value; only the tensor maps have an address that matters.
template <int HD, int F>
__device__ __noinline__ void dkv_call(uint32_t tmem, const DkvMaps& tm, const BwdArgs a, const KernelGuard guard) {
  dkv_pass<HD, F>(Shared<HD>::keys(), Shared<HD>::base(), tmem, tm, a, guard);
}
template <int HD, int F>
__device__ __noinline__ void dq_call(uint32_t tmem, const DqMaps& tm, const BwdArgs a, const KernelGuard guard) {
  dq_pass<HD, F>(Shared<HD>::queries(), Shared<HD>::base(), tmem, tm, a, guard);
}

// One launch for both passes: nothing is read before the wait at its start, which orders everything either
// pass reads after the preparation and all before it, and a pair that has no more key items goes on with its
// query items at once.  4608 x 32 heads of 128 in f16: 905 us, seven products at 1345 TFLOP/s and 1.54 GHz, the
// tensor core busy in 72 % of the cycles.  Two launches, the second waiting for all of the first: 1100 tokens x
// 16 heads of 128 66 us against 54, 80 tokens x 4 heads of 64 13.7 against 9.6, the padded batch of 16 heads of 64
// 151 against 146; 4608 x 32 heads of 128 in bf16 852 against 861.
template <int HD, int F>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Shared<HD>::THREADS, 1)
    bwd_kernel(const __grid_constant__ BwdMaps tm, const __grid_constant__ BwdArgs a, const KernelGuard guard) {
  using S = Shared<HD>;
  if (threadIdx.x == 0) {
    S::keys().init();
    S::queries().init();
  }
  uint32_t* tmem_slot = S::keys().tmem_slot;
  if (warp_id() == 2) tmem_alloc_pair(tmem_slot, TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers exist before any remote arrive or TMA
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (threadIdx.x < sizeof(tm) / sizeof(CUtensorMap))
    tma_prefetch_desc(reinterpret_cast<const CUtensorMap*>(&tm) + threadIdx.x);
  pdl_wait_then_release();
  dkv_call<HD, F>(tmem, tm.dkv, a, guard);
  // the key pass's copies have landed, its products retired and its boxes left shared memory
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  dq_call<HD, F>(tmem, tm.dq, a, guard);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA leaves while the pair MMAs or remote arrives may touch it
  if (warp_id() == 2) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, TMEM_COLS);
  }
}

// ------------------------------------------------------------------ launch

static bool map_rows(CUtensorMap* m, int fmt, const void* p, int64_t ld, int rows, int batch, int cols, int box_cols,
                     int box_rows, bool plain = false) {
  const uint64_t dims[3] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(rows), static_cast<uint64_t>(batch)};
  const uint64_t strides[2] = {static_cast<uint64_t>(ld) * 2, static_cast<uint64_t>(rows) * ld * 2};
  const uint32_t box[3] = {static_cast<uint32_t>(box_cols), static_cast<uint32_t>(box_rows), 1};
  return make_tmap(m, fmt == FMT_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                   const_cast<void*>(p), dims, strides, box,
                   plain            ? CU_TENSOR_MAP_SWIZZLE_NONE
                   : box_cols == 32 ? CU_TENSOR_MAP_SWIZZLE_64B
                                    : CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int HD, int F>
static cudaError_t launch_hd(Rows q, Rows k, Rows v, const void* out, const void* dout, const float* lse, Rows dq,
                             Rows dk, Rows dv, int batch, int seq, int n_heads, const int32_t* key_lens,
                             void* workspace, const KernelGuard& g, cudaStream_t s) {
  using LQ = DqLayout<HD>;
  using LK = DkvLayout<HD>;
  const Workspace w = carve(workspace, batch, seq, n_heads, HD);
  const int d = n_heads * HD, nblk = blocks_of(seq) + 1;
  const size_t one = static_cast<size_t>(batch) * T * d;
  const Rows go{dout, d}, tq{w.tails, d}, tk{w.tails + one, d}, tdo{w.tails + 2 * one, d};
  bool ok = true;
  auto tile = [&](CUtensorMap* m, Rows r) { ok = ok && map_rows(m, F, r.p, r.ld, seq, batch, d, 64, T); };
  // the two cuts of a block of `blk` rows
  auto cuts = [&](CUtensorMap* by_rows, CUtensorMap* by_cols, Rows r, int n, int blk) {
    ok = ok && map_rows(by_rows, F, r.p, r.ld, n, batch, d, 64, blk / 2);
    if (by_cols != nullptr) ok = ok && map_rows(by_cols, F, r.p, r.ld, n, batch, d, HD / 2, blk);
  };
  BwdMaps maps = {};
  DqMaps& mq = maps.dq;
  tile(&mq.q, q);
  tile(&mq.dout, go);
  cuts(&mq.k_rows, &mq.k_cols, k, seq, LQ::R);
  cuts(&mq.v_rows, nullptr, v, seq, LQ::R);
  if (key_lens != nullptr) {
    cuts(&mq.tk_rows, &mq.tk_cols, tk, T, LQ::R);
  } else {  // no other call reads a tail
    mq.tk_rows = mq.k_rows;
    mq.tk_cols = mq.k_cols;
  }
  DkvMaps& mk = maps.dkv;
  tile(&mk.k, k);
  tile(&mk.v, v);
  cuts(&mk.q_rows, &mk.q_cols, q, seq, LK::R);
  cuts(&mk.do_rows, &mk.do_cols, go, seq, LK::R);
  if (key_lens != nullptr) {
    cuts(&mk.tq_rows, &mk.tq_cols, tq, T, LK::R);
    cuts(&mk.tdo_rows, &mk.tdo_cols, tdo, T, LK::R);
  } else {
    mk.tq_rows = mk.q_rows;
    mk.tq_cols = mk.q_cols;
    mk.tdo_rows = mk.do_rows;
    mk.tdo_cols = mk.do_cols;
  }
  // boxes of 32 rows x OUT columns, unswizzled
  auto out_map = [&](CUtensorMap* m, Rows r, int cols) { ok = ok && map_rows(m, F, r.p, r.ld, seq, batch, d, cols, 32, true); };
  out_map(&mq.dq, dq, LQ::OUT);
  out_map(&mk.dk, dk, LK::OUT);
  out_map(&mk.dv, dv, LK::OUT);
  if (!ok) return cudaErrorInvalidValue;
  cudaError_t e = allow_smem<bwd_kernel<HD, F>>(Shared<HD>::SMEM);
  if (e != cudaSuccess) return e;
  const PrepArgs pa{static_cast<const uint16_t*>(q.p), static_cast<const uint16_t*>(k.p),
                    static_cast<const uint16_t*>(v.p), static_cast<const uint16_t*>(out),
                    static_cast<const uint16_t*>(dout), q.ld, k.ld, v.ld, lse, key_lens, w.nlse2, w.ndelta, w.rows2,
                    w.norms2, w.tails, batch, seq, n_heads};
  e = launch_pdl(bwd_prep_kernel<HD, F>, dim3(nblk, n_heads, batch), dim3(PREP_THREADS), 0, s, pa);
  if (e != cudaSuccess) return e;
  int sms = 0, dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    sms = 148;
  auto view = [](Rows r) { return OutRows{static_cast<uint16_t*>(const_cast<void*>(r.p)), r.ld}; };
  const BwdArgs args{w.nlse2, w.ndelta, w.rows2, w.norms2, view(dq), view(dk), view(dv), key_lens, batch, seq, n_heads};
  const int64_t items = static_cast<int64_t>((seq + 2 * T - 1) / (2 * T)) * n_heads * batch, pairs = sms / 2;
  const dim3 grid(2u * static_cast<unsigned>(2 * items < pairs ? 2 * items : pairs));
  return launch_pdl(bwd_kernel<HD, F>, grid, dim3(Shared<HD>::THREADS), Shared<HD>::SMEM, s, maps, args, g);
}

}  // namespace abwd

size_t attention_bwd_workspace(int batch, int seq, int n_heads, int head_dim) {
  return abwd::carve(nullptr, batch, seq, n_heads, head_dim).bytes;
}

cudaError_t launch_attention_bwd(Rows q, Rows k, Rows v, const void* out, const void* dout, const float* lse, Rows dq,
                                 Rows dk, Rows dv, int fmt, int batch, int seq, int n_heads, int head_dim,
                                 const int32_t* key_lens, void* workspace, const KernelGuard& g, cudaStream_t s) {
  auto run = [&](auto fn) {
    return fn(q, k, v, out, dout, lse, dq, dk, dv, batch, seq, n_heads, key_lens, workspace, g, s);
  };
  if (head_dim == 128)
    return fmt == FMT_F16 ? run(abwd::launch_hd<128, FMT_F16>) : run(abwd::launch_hd<128, FMT_BF16>);
  if (head_dim == 64) return fmt == FMT_F16 ? run(abwd::launch_hd<64, FMT_F16>) : run(abwd::launch_hd<64, FMT_BF16>);
  return cudaErrorInvalidValue;
}

}  // namespace jab
