// The gradient of the joint attention (Ideogram 4 deep dive, section 4-2: one sequence, one
// bidirectional self-attention), the probabilities recomputed from q, k and the row log-sum-exps:
//   P = exp(q k^T / sqrt(hd) - lse)         delta_q = sum_c dO_qc O_qc
//   dV = P^T dO     dP = dO V^T     dS = P o (dP - delta) / sqrt(hd)     dQ = dS K     dK = dS^T Q
// Three launches:
//   bwd_prep_kernel  delta and the row log-sum-exps in log2 units, padded to whole blocks of 128
//                    rows, and what the other two need to know of the data (see below)
//   bwd_dq_kernel    256 queries per CTA pair, over all key blocks
//   bwd_dkv_kernel   256 keys per CTA pair, over all query blocks
// S and dP are computed in both of the latter, seven products instead of five: dQ is summed over
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
// (P <= 1), dS by the sigma below, both undone on the fp32 accumulators.  With
// A = max_q |dO_q| and B = max_k |V_k| (Euclidean norms over one head's channels),
// |dP - delta| <= 2 A B, so sigma = 2^floor(14 - log2(2 A B)) keeps every |dS| below 2^15.
#include "common.cuh"
#include "pipeline.cuh"
#include "train.h"

namespace jab {
namespace abwd {

constexpr int T = 128;   // rows of an own tile per CTA; keys of a block in dq
constexpr int BQ = 96;   // queries of a block in dkv
constexpr int COLS = 32;  // columns of a block per elementwise thread: a warp for each 32 x 32 piece
constexpr int TMEM_COLS = 512;
constexpr float LOG2E = 1.4426950408889634f;
constexpr float P_SHIFT = 15.f;  // f16: P is held as 2^15 P

__host__ __device__ inline int blocks_of(int seq) { return (seq + T - 1) / T; }

// Per (b, h), nblk = the blocks of 128 rows and one more (blocks of 96 rows end inside it):
// ws.lse2 / ws.delta [B, H, nblk * 128]; norms2 [B, H, nblk]: the block's max |dO_q|^2 and
// max |V_k|^2 (f16 only); tails: zero-padded copies [3: q, k, dO][B, 128, H hd].
struct Workspace {
  float* lse2;
  float* delta;
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
  w.lse2 = reinterpret_cast<float*>(b);
  w.delta = reinterpret_cast<float*>(b + vec);
  w.norms2 = reinterpret_cast<float2*>(b + 2 * vec);
  w.tails = reinterpret_cast<uint16_t*>(b + 2 * vec + nrm);
  w.bytes = 2 * vec + nrm + tail;
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
  float *lse2, *delta;
  float2* norms2;
  uint16_t* tails;
  int batch, seq, n_heads;
};

// One CTA per (block of 128 rows, head, element); HD / 8 lanes per row.  HBM-bound: reads O and dO
// (f16: and V) once.
template <int HD, int F>
__global__ void __launch_bounds__(256) bwd_prep_kernel(const PrepArgs a) {
  constexpr int LANES = HD / 8;
  constexpr int ROWS = 256 / LANES;
  constexpr int PASSES = T / ROWS;
  __shared__ float2 red[8];
  pdl_wait_then_release();
  const int blk = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int nblk = gridDim.x;
  const int n = tokens_of(a.key_lens, b, a.seq);
  const int d = a.n_heads * HD;
  const int c = static_cast<int>(threadIdx.x) % LANES, r0 = static_cast<int>(threadIdx.x) / LANES;
  const int64_t bh = static_cast<int64_t>(b) * a.n_heads + h;
  float* lse2 = a.lse2 + (bh * nblk + blk) * T;
  float* delta = a.delta + (bh * nblk + blk) * T;
  float mdo = 0.f, mv = 0.f;
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    const int r = p * ROWS + r0;
    const int row = blk * T + r;
    float dot = 0.f, sdo = 0.f, sv = 0.f;
    if (row < n) {
      const int64_t at = (static_cast<int64_t>(b) * a.seq + row);
      float o[8], g[8];
      load8<F>(a.o + at * d + h * HD, c, o);
      load8<F>(a.dout + at * d + h * HD, c, g);
#pragma unroll
      for (int k = 0; k < 8; ++k) dot = fmaf(o[k], g[k], dot);
      if constexpr (F == FMT_F16) {
        float v[8];
        load8<F>(a.v + at * a.ldv + h * HD, c, v);
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
      delta[r] = dot;
      lse2[r] = row < n ? a.lse[bh * a.seq + row] * LOG2E - (F == FMT_F16 ? P_SHIFT : 0.f) : INFINITY;
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
      for (int w = 1; w < 8; ++w) {
        mdo = fmaxf(mdo, red[w].x);
        mv = fmaxf(mv, red[w].y);
      }
      a.norms2[bh * nblk + blk] = make_float2(mdo, mv);
    }
  }
  // k: the block of 128 rows in which the tokens end; q and dO: the block of 96
  const bool tk = has_tail(n, a.seq, T) && blk == n / T;
  const int q0 = n / BQ * BQ;
  const bool tq = has_tail(n, a.seq, BQ) && blk * T < q0 + BQ && blk * T + T > q0;
  if (tk || tq) {
    const size_t one = static_cast<size_t>(a.batch) * T * d;
    for (int p = 0; p < PASSES; ++p) {
      const int r = p * ROWS + r0;
      const int row = blk * T + r;
      const int64_t at = static_cast<int64_t>(b) * a.seq + row;
      auto put = [&](const uint16_t* src, int64_t ld, int which, int dst_row) {
        const uint4 x = row < n ? reinterpret_cast<const uint4*>(src + at * ld + h * HD)[c] : make_uint4(0u, 0u, 0u, 0u);
        reinterpret_cast<uint4*>(a.tails + which * one + (static_cast<size_t>(b) * T + dst_row) * d + h * HD)[c] = x;
      };
      if (tk) put(a.k, a.ldk, 1, r);
      if (tq && row >= q0 && row < q0 + BQ) {
        put(a.q, a.ldq, 0, row - q0);
        put(a.dout, d, 2, row - q0);
      }
    }
  }
}

// log2 of the factor dS is multiplied by before its rounding to f16 (0 in bf16, whose exponent
// range is fp32's): 14 - log2(2 A B) rounded down, from the per-block maxima.  Norms of zero, or
// ones that are not finite, leave it at 0.  Every lane of a warp calls it.
template <int F>
__device__ __forceinline__ float ds_shift(const float2* norms2, int nblk) {
  if constexpr (F != FMT_F16) return 0.f;
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
  // 2 A B = 2 sqrt(a b); the sum of logs cannot overflow
  const float l = 1.f + 0.5f * (log2f(a) + log2f(b));
  return l > -100.f && l < 100.f ? floorf(14.f - l) : 0.f;
}

// Shared memory of one CTA.  Own tiles: 128 rows x HD (K and V in dkv, Q and dO in dq), slabs of 64
// columns, 128-byte swizzle.  Ring slots hold this CTA's half of a block of R rows of the other axis,
// in one of two cuts of the same size: "rows", R / 2 rows x HD, the B operand of a product over HD, or
// "cols", R rows x HD / 2, the B operand of a product over the rows.
template <int HD, int R, int RINGS>
struct Layout {
  static constexpr int N = 3;  // slots of a ring
  static constexpr int PARTS = R / COLS;
  static constexpr int EW_WARPS = 4 * PARTS;
  static constexpr int THREADS = 64 + 32 * EW_WARPS;
  static constexpr int SLAB = T * 128;
  static constexpr int TILE = (HD / 64) * SLAB;
  static constexpr int RSLAB = R / 2 * 128;
  static constexpr int CUT = R * HD;  // bytes of one ring slot, either cut
  static constexpr int OFF_A = 0;
  static constexpr int OFF_B = OFF_A + TILE;
  static constexpr int OFF_RING = OFF_B + TILE;
  static constexpr int OFF_VEC = OFF_RING + RINGS * N * CUT;  // dkv: [N][lse2 | delta], R each
  static constexpr int OFF_BAR = OFF_VEC + N * 2 * R * 4;
  static constexpr int NUM_BARS = 48;
  static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;
  static constexpr int SMEM = OFF_MISC + 16 + 1024;
  static_assert(SMEM <= 232448, "227 KB of shared memory per CTA");
  static_assert(RSLAB % 1024 == 0 && CUT % 1024 == 0, "swizzled tiles keep their alignment");
};

// Global -> shared copy of a multiple of 16 bytes, both addresses 16-byte aligned.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

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
    tma_load_3d_pair(dst + c * L::RSLAB, m, bar, x + 64 * c, y + L::RSLAB / 128 * rank, z);
}
template <int HD>
__device__ __forceinline__ void load_cols_cut(uint8_t* dst, const CUtensorMap* m, uint32_t bar, int x, int y, int z,
                                              int rank) {
  tma_load_3d_pair(dst, m, bar, x + rank * (HD / 2), y, z);
}

// The descriptor of the same layout `bytes` further on.  One 32-bit add: the start address (in 16-byte
// units) fills the low 14 bits and stays below 2^14 inside 227 KB.  Building each descriptor from its
// address instead made the issuing lane the slowest part of the kernel (about 110 clocks per MMA).
__device__ __forceinline__ uint64_t desc_at(uint64_t d, uint32_t bytes) {
  return (d & 0xFFFFFFFF00000000ull) | (static_cast<uint32_t>(d) + (bytes >> 4));
}

// D[256 x R] = A B^T over HD: A both CTAs' own tiles, B a block in the rows cut.
template <class L, int HD, int F>
__device__ __forceinline__ void mma_rows(uint32_t d, const uint8_t* a, const uint8_t* b) {
  constexpr uint32_t idesc = idesc_f16kind(2 * T, L::RSLAB / 64, F == FMT_F16, false, false);
  const uint64_t ad = smem_desc_sw128(smem_u32(a), 16, 1024), bd = smem_desc_sw128(smem_u32(b), 16, 1024);
#pragma unroll
  for (int kk = 0; kk < HD / 16; ++kk) {
    constexpr int RS = L::RSLAB, AS = L::SLAB;
    mma_f16kind_ss_pair(d, desc_at(ad, (kk >> 2) * AS + (kk & 3) * 32), desc_at(bd, (kk >> 2) * RS + (kk & 3) * 32),
                        idesc, kk > 0 ? 1u : 0u);
  }
}

// D[256 x HD] (+)= A[256 x R] B: A as 16-bit pairs in TMEM, 16 columns for every COLS = 32 values and
// those pieces `step` columns apart; B a block in the cols cut, its rows being the contraction axis.
template <int R, int HD, int F>
__device__ __forceinline__ void mma_cols(uint32_t d, uint32_t a, int step, const uint8_t* b, bool accumulate) {
  constexpr uint32_t idesc = idesc_f16kind(2 * T, HD, F == FMT_F16, false, true);
  const uint64_t bd = HD == 128 ? smem_desc_sw128(smem_u32(b), 16, 8 * HD) : smem_desc_sw64(smem_u32(b), 16, 8 * HD);
#pragma unroll
  for (int kk = 0; kk < R / 16; ++kk)  // 16 rows of HD / 2 values
    mma_f16kind_ts_pair(d, a + step * (kk >> 1) + 8 * (kk & 1), desc_at(bd, kk * 16 * HD), idesc,
                        (accumulate || kk > 0) ? 1u : 0u);
}

__device__ __forceinline__ void get_part(uint32_t taddr, float (&v)[COLS]) {
  static_assert(COLS == 32, "one TMEM load");
  uint32_t a[32];
  tmem_ld32(taddr, a);
  tmem_ld_wait_regs(a);
#pragma unroll
  for (int k = 0; k < COLS; ++k) v[k] = __uint_as_float(a[k]);
}

// A thread's values as 16-bit pairs into COLS / 2 columns.
template <int F>
__device__ __forceinline__ void put_part(uint32_t taddr, const float (&v)[COLS]) {
  uint32_t pk[COLS / 2];
#pragma unroll
  for (int k = 0; k < COLS / 2; ++k) pk[k] = pack2<F>(v[2 * k], v[2 * k + 1]);
  tmem_st16(taddr, pk);
  tmem_st_wait();
}

// NC columns of one accumulator row (fp32 at taddr) times f into a 16-bit row, or zeros.
template <int NC, int F>
__device__ __forceinline__ void store_row(uint32_t taddr, float f, uint16_t* dst, bool in_range, bool live) {
#pragma unroll
  for (int c = 0; c < NC / 32; ++c) {
    uint32_t raw[32];
    tmem_ld32(taddr + 32 * c, raw);
    tmem_ld_wait_regs(raw);
    if (in_range) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float o[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = live ? __uint_as_float(raw[8 * q + k]) * f : 0.f;
        store8<F>(dst + 32 * c, q, o);
      }
    }
  }
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
    return mbar_wait(&empty[slot(u)], phase(u) ^ 1u, g, abort_flag, where);
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
__device__ __forceinline__ Item item_of(int i, int ntile, int n_heads, int seq, const int32_t* key_lens, int rows) {
  Item it;
  it.tt = i % ntile;
  it.bh = i / ntile;
  it.head = static_cast<int>(it.bh % n_heads);
  it.b = static_cast<int>(it.bh / n_heads);
  it.n = tokens_of(key_lens, it.b, seq);
  it.nb = it.tt * 2 * T < it.n ? (it.n + rows - 1) / rows : 0;
  return it;
}

// ------------------------------------------------------------------ dK, dV

// Two CTAs on two SMs (a cluster) share 256 keys of one head, 128 each, and walk the queries in blocks
// of 96; the pair MMA (cta_group::2, M = 256) lets each CTA hold half of every query block.  The
// products run with the keys as rows (S^T = K Q^T, dP^T = V dO^T), so that P^T and dS^T come out of the
// elementwise step in the layout in which the tensor core reads an A operand from TMEM:
// dV += P^T dO, dK += dS^T Q.
// TMEM of each CTA: S^T 96 | dP^T 96 | P^T 48 | (16 unused) | dV | dK, 128 columns each; dS^T overwrites
// dP^T as 16-bit pairs.  With blocks of 128 queries P^T has no columns of its own and must overwrite
// S^T, so S(j+1) waits for dV(j), which waits for the whole exponential step of block j: 3420 clocks per
// block of 128 against the products' 2048.  With 96, S(j+1) runs as soon as S(j) has been read into
// registers and the elementwise warps never wait for it.
// Persistent: pair p takes work items p, p + pairs, ...; rings and barrier phases run on across items.
//   warp 0       loads.  Q and dO of a block come in both cuts, each with a ring of its own, since
//                S frees Q's rows long before dK frees its columns
//   warp 1       TMEM; in the leader one lane issues S(j+1) when S(j) has been read, dV(j) when P(j) is
//                written, dK(j) and dP(j+1) when dS(j) is
//   warps 2..13  P^T = exp2(c S^T - lse2), then dS^T = P^T (dP^T - delta); thread = key row and a third
//                of the query columns; at the end of an item the rows of dV and dK.
struct DkvMaps {
  CUtensorMap k, v, q_rows, q_cols, do_rows, do_cols, tq_rows, tq_cols, tdo_rows, tdo_cols;
};
template <int HD>
using DkvLayout = Layout<HD, BQ, 4>;

template <int HD, int F>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(DkvLayout<HD>::THREADS, 1)
    bwd_dkv_kernel(const __grid_constant__ DkvMaps tm, const float* __restrict__ lse2, const float* __restrict__ delta,
                   const float2* __restrict__ norms2, OutRows dk, OutRows dv, int batch, int seq, int n_heads,
                   const int32_t* __restrict__ key_lens, const KernelGuard guard) {
  using L = DkvLayout<HD>;
  constexpr int N = L::N;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sK = smem + L::OFF_A;
  uint8_t* sV = smem + L::OFF_B;
  uint8_t* sQr = smem + L::OFF_RING;
  uint8_t* sOr = sQr + N * L::CUT;
  uint8_t* sOc = sOr + N * L::CUT;
  uint8_t* sQc = sOc + N * L::CUT;
  float* sVec = reinterpret_cast<float*>(smem + L::OFF_VEC);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  const Ring<N> qr(bars), dor(bars + 2 * N), doc(bars + 4 * N), qc(bars + 6 * N);
  const Ring<1> kt(bars + 8 * N), vt(bars + 8 * N + 2);
  uint64_t* vec_full = bars + 8 * N + 4;  // [N] this CTA's copies
  uint64_t* vec_empty = vec_full + N;     // [N] the elementwise warps of this CTA
  uint64_t* s_full = vec_empty + N;
  uint64_t* s_empty = s_full + 1;          // leader: every elementwise warp of both CTAs
  uint64_t* dp_full = s_empty + 1;
  uint64_t* p_full = dp_full + 1;          // leader: every elementwise warp of both CTAs
  uint64_t* p_empty = p_full + 1;          // dV has read P
  uint64_t* ds_full = p_empty + 1;         // leader: every elementwise warp of both CTAs
  uint64_t* acc_full = ds_full + 1;
  uint64_t* acc_empty = acc_full + 1;      // leader: every elementwise warp of both CTAs
  uint64_t* drain_bar = acc_empty + 1;
  static_assert(8 * N + 4 + 2 * N + 9 <= L::NUM_BARS, "barriers fit");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + L::OFF_MISC + 4);

  const int warp = static_cast<int>(warp_id());
  const int lane = static_cast<int>(lane_id());
  const int rank = static_cast<int>(cluster_ctarank());
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int nblk = blocks_of(seq) + 1;
  const int ntile = (seq + 2 * T - 1) / (2 * T);
  const int items = batch * n_heads * ntile;

  if (threadIdx.x == 0) {
    qr.init();
    dor.init();
    doc.init();
    qc.init();
    kt.init();
    vt.init();
    for (int i = 0; i < N; ++i) {
      mbar_init(&vec_full[i], 1);
      mbar_init(&vec_empty[i], L::EW_WARPS);
    }
    mbar_init(s_full, 1);
    mbar_init(s_empty, 2 * L::EW_WARPS);
    mbar_init(dp_full, 1);
    mbar_init(p_full, 2 * L::EW_WARPS);
    mbar_init(p_empty, 1);
    mbar_init(ds_full, 2 * L::EW_WARPS);
    mbar_init(acc_full, 1);
    mbar_init(acc_empty, 2 * L::EW_WARPS);
    mbar_init(drain_bar, 1);
    *abort_flag = 0u;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc_pair(tmem_slot, TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers exist before any remote arrive or TMA
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t t_s = tmem, t_dp = tmem + 96, t_p = tmem + 192, t_dv = tmem + 256, t_dk = tmem + 384;
  pdl_wait_then_release();

  if (warp == 0) {
    const bool one = elect_one();
    int u = 0, ui = 0;
    int n_qr = 0, n_or = 0, n_oc = 0, n_qc = 0, n_k = 0, n_v = 0, n_vec = 0;
    bool ok = true;
    auto where = [&](int i) { return where_code(ERR_TIMEOUT_ABWD_PRODUCER, rank, i); };
    for (int i = pair; i < items && ok; i += pairs) {
      const Item it = item_of(i, ntile, n_heads, seq, key_lens, BQ);
      if (it.nb == 0) continue;
      const bool tail = has_tail(it.n, seq, BQ);
      const int x = it.head * HD, row0 = it.tt * 2 * T + rank * T;
      ok = kt.wait_empty(ui, guard, abort_flag, where(0xFFFF));
      if (!ok) break;
      if (one) load_tile<L, HD>(sK, &tm.k, kt.arm(ui, leader, 2 * L::TILE), x, row0, it.b);
      ++n_k;
      __syncwarp();
      for (int j = 0; j < it.nb; ++j, ++u) {
        const bool tl = tail && j == it.nb - 1;
        const int y = tl ? 0 : j * BQ, st = u % N;
        ok = qr.wait_empty(u, guard, abort_flag, where(u));
        if (!ok) break;
        if (one)
          load_rows_cut<L, HD>(sQr + st * L::CUT, tl ? &tm.tq_rows : &tm.q_rows, qr.arm(u, leader, 2 * L::CUT), x, y,
                               it.b, rank);
        ++n_qr;
        __syncwarp();
        ok = mbar_wait(&vec_empty[st], (static_cast<uint32_t>(u / N) & 1u) ^ 1u, guard, abort_flag, where(u));
        if (!ok) break;
        if (one) {
          float* vec = sVec + st * 2 * BQ;
          mbar_arrive_expect_tx(&vec_full[st], 2 * BQ * 4);
          bulk_load(vec, lse2 + it.bh * nblk * T + j * BQ, BQ * 4, &vec_full[st]);
          bulk_load(vec + BQ, delta + it.bh * nblk * T + j * BQ, BQ * 4, &vec_full[st]);
        }
        ++n_vec;
        __syncwarp();
        if (j == 0) {
          ok = vt.wait_empty(ui, guard, abort_flag, where(0xFFFE));
          if (!ok) break;
          if (one) load_tile<L, HD>(sV, &tm.v, vt.arm(ui, leader, 2 * L::TILE), x, row0, it.b);
          ++n_v;
          __syncwarp();
        }
        ok = dor.wait_empty(u, guard, abort_flag, where(u));
        if (!ok) break;
        if (one)
          load_rows_cut<L, HD>(sOr + st * L::CUT, tl ? &tm.tdo_rows : &tm.do_rows, dor.arm(u, leader, 2 * L::CUT), x, y,
                               it.b, rank);
        ++n_or;
        __syncwarp();
        ok = doc.wait_empty(u, guard, abort_flag, where(u));
        if (!ok) break;
        if (one)
          load_cols_cut<HD>(sOc + st * L::CUT, tl ? &tm.tdo_cols : &tm.do_cols, doc.arm(u, leader, 2 * L::CUT), x, y,
                            it.b, rank);
        ++n_oc;
        __syncwarp();
        ok = qc.wait_empty(u, guard, abort_flag, where(u));
        if (!ok) break;
        if (one)
          load_cols_cut<HD>(sQc + st * L::CUT, tl ? &tm.tq_cols : &tm.q_cols, qc.arm(u, leader, 2 * L::CUT), x, y, it.b,
                            rank);
        ++n_qc;
        __syncwarp();
      }
      ++ui;
    }
    // Never leave with copies in flight: the leader's barriers count both CTAs' copies, and the peer is
    // held by the final cluster barrier until the leader has drained.
    const uint32_t wd = where_code(ERR_TIMEOUT_ABWD_DRAIN, rank, 0);
    for (int v = n_vec > N ? n_vec - N : 0; v < n_vec; ++v)
      mbar_wait(&vec_full[v % N], static_cast<uint32_t>(v / N) & 1u, guard, abort_flag, wd, true);
    if (leader) {
      kt.drain(n_k, guard, abort_flag, wd);
      vt.drain(n_v, guard, abort_flag, wd);
      qr.drain(n_qr, guard, abort_flag, wd);
      dor.drain(n_or, guard, abort_flag, wd);
      doc.drain(n_oc, guard, abort_flag, wd);
      qc.drain(n_qc, guard, abort_flag, wd);
    }
  } else if (warp == 1) {
    const bool one = elect_one();
    if (leader) {
      auto where = [&](int k, int i) { return where_code(ERR_TIMEOUT_ABWD_MMA, k, i); };
      // S(u) overwrites S(u - 1) once every warp has read it
      auto issue_s = [&](int u, bool last) {
        if (!qr.wait_full(u, guard, abort_flag, where(0, u)) ||
            (u > 0 && !mbar_wait(s_empty, static_cast<uint32_t>(u - 1) & 1u, guard, abort_flag, where(1, u))))
          return false;
        tc_fence_after();
        if (one) {
          mma_rows<L, HD, F>(t_s, sK, sQr + (u % N) * L::CUT);
          mma_commit_pair(s_full, 0x3);
          mma_commit_pair(&qr.empty[u % N], 0x3);
          if (last) mma_commit_pair(&kt.empty[0], 0x3);
        }
        __syncwarp();
        return true;
      };
      // dP(u) overwrites dS(u - 1), which dK(u - 1), issued before, has read by then (in-order issue)
      auto issue_dp = [&](int u, bool last) {
        if (!dor.wait_full(u, guard, abort_flag, where(2, u))) return false;
        tc_fence_after();
        if (one) {
          mma_rows<L, HD, F>(t_dp, sV, sOr + (u % N) * L::CUT);
          mma_commit_pair(dp_full, 0x3);
          mma_commit_pair(&dor.empty[u % N], 0x3);
          if (last) mma_commit_pair(&vt.empty[0], 0x3);
        }
        __syncwarp();
        return true;
      };
      bool ok = true;
      int u = 0, ui = 0;
      for (int i = pair; i < items && ok; i += pairs) {
        const int nb = item_of(i, ntile, n_heads, seq, key_lens, BQ).nb;
        if (nb == 0) continue;
        ok = kt.wait_full(ui, guard, abort_flag, where(3, u)) && issue_s(u, nb == 1) &&
             vt.wait_full(ui, guard, abort_flag, where(4, u)) && issue_dp(u, nb == 1);
        for (int j = 0; j < nb && ok; ++j, ++u) {
          const bool next = j + 1 < nb;
          const uint32_t par = static_cast<uint32_t>(u) & 1u;
          // the first dV of an item overwrites accumulators that both CTAs must have read
          ok = (!next || issue_s(u + 1, j + 2 == nb)) && doc.wait_full(u, guard, abort_flag, where(5, u)) &&
               (j > 0 || ui == 0 ||
                mbar_wait(acc_empty, static_cast<uint32_t>(ui - 1) & 1u, guard, abort_flag, where(6, u))) &&
               mbar_wait(p_full, par, guard, abort_flag, where(7, u));
          if (!ok) break;
          tc_fence_after();
          if (one) {
            mma_cols<BQ, HD, F>(t_dv, t_p, COLS / 2, sOc + (u % N) * L::CUT, j > 0);
            mma_commit_pair(p_empty, 0x3);
            mma_commit_pair(&doc.empty[u % N], 0x3);
          }
          __syncwarp();
          ok = qc.wait_full(u, guard, abort_flag, where(8, u)) && mbar_wait(ds_full, par, guard, abort_flag, where(9, u));
          if (!ok) break;
          tc_fence_after();
          if (one) {
            mma_cols<BQ, HD, F>(t_dk, t_dp, COLS, sQc + (u % N) * L::CUT, j > 0);
            mma_commit_pair(&qc.empty[u % N], 0x3);
          }
          __syncwarp();
          if (next) ok = issue_dp(u + 1, j + 2 == nb);
        }
        if (ok && one) mma_commit_pair(acc_full, 0x3);
        __syncwarp();
        ++ui;
      }
      if (one) mma_commit_pair(drain_bar, 0x3);  // all MMAs retired before either CTA frees TMEM
      __syncwarp();
    }
    mbar_wait(drain_bar, 0u, guard, abort_flag, where_code(ERR_TIMEOUT_ABWD_DRAIN, rank, 1), true);
  } else {
    const int part = (warp - 2) >> 2;
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t s_col = t_s + lane_off + COLS * part;
    const uint32_t dp_col = t_dp + lane_off + COLS * part;
    const uint32_t p_col = t_p + lane_off + COLS / 2 * part;
    const float scale = HD == 128 ? 0.08838834764831845f : 0.125f;
    const float2 c2 = make_float2(scale * LOG2E, scale * LOG2E);
    auto where = [&](int k, int i) { return where_code(ERR_TIMEOUT_ABWD_SOFTMAX, k, i); };
    bool ok = true;
    int u = 0, ui = 0;
    for (int i = pair; i < items && ok; i += pairs) {
      const Item it = item_of(i, ntile, n_heads, seq, key_lens, BQ);
      const int row0 = it.tt * 2 * T + rank * T;
      if (it.nb == 0) {
        const int t = static_cast<int>(threadIdx.x) - 64;
        zero_rows<HD, 32 * L::EW_WARPS>(dk.p + static_cast<int64_t>(it.b) * seq * dk.ld + it.head * HD, dk.ld, row0, seq, t);
        zero_rows<HD, 32 * L::EW_WARPS>(dv.p + static_cast<int64_t>(it.b) * seq * dv.ld + it.head * HD, dv.ld, row0, seq, t);
        continue;
      }
      const float shift = ds_shift<F>(norms2 + it.bh * nblk, blocks_of(it.n));
      // P carries 2^15 in f16; dS = that P times (dP - delta) times tau = 2^(shift - 15)
      const float tau = F == FMT_F16 ? exp2f(shift - P_SHIFT) : 1.f;
      for (int j = 0; j < it.nb; ++j, ++u) {
        const uint32_t par = static_cast<uint32_t>(u) & 1u;
        const int st = u % N;
        const float* vec = sVec + st * 2 * BQ + COLS * part;
        ok = mbar_wait(&vec_full[st], static_cast<uint32_t>(u / N) & 1u, guard, abort_flag, where(0, u)) &&
             mbar_wait(s_full, par, guard, abort_flag, where(1, u));
        if (!ok) break;
        tc_fence_after();
        float p[COLS];
        get_part(s_col, p);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(mapa_shared(smem_u32(s_empty), 0));
#pragma unroll
        for (int k = 0; k < COLS; k += 2) {
          const float2 l = *reinterpret_cast<const float2*>(vec + k);
          const float2 x = fma2(make_float2(p[k], p[k + 1]), c2, make_float2(-l.x, -l.y));
          p[k] = ex2_approx(x.x);
          p[k + 1] = ex2_approx(x.y);
        }
        ok = mbar_wait(p_empty, par ^ 1u, guard, abort_flag, where(2, u));
        if (!ok) break;
        tc_fence_after();
        put_part<F>(p_col, p);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(mapa_shared(smem_u32(p_full), 0));
        ok = mbar_wait(dp_full, par, guard, abort_flag, where(3, u));
        if (!ok) break;
        tc_fence_after();
        float x[COLS];
        get_part(dp_col, x);
#pragma unroll
        for (int k = 0; k < COLS; k += 2) {
          const float2 dl = *reinterpret_cast<const float2*>(vec + BQ + k);
          float2 y = add2(make_float2(x[k], x[k + 1]), make_float2(-dl.x, -dl.y));
          y = mul2(y, make_float2(p[k], p[k + 1]));
          if constexpr (F == FMT_F16) y = mul2(y, make_float2(tau, tau));
          x[k] = y.x;
          x[k + 1] = y.y;
        }
        put_part<F>(dp_col, x);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&vec_empty[st]);
          mbar_arrive_remote(mapa_shared(smem_u32(ds_full), 0));
        }
      }
      if (!ok) break;
      ok = mbar_wait(acc_full, static_cast<uint32_t>(ui) & 1u, guard, abort_flag, where(4, u));
      if (!ok) break;
      tc_fence_after();
      {
        // 2 HD / 32 pieces of 32 columns (dV's, then dK's), dealt to the row's warps in turn
        const int row = row0 + r;
        uint16_t* dst_v = dv.p + (static_cast<int64_t>(it.b) * seq + row) * dv.ld + it.head * HD;
        uint16_t* dst_k = dk.p + (static_cast<int64_t>(it.b) * seq + row) * dk.ld + it.head * HD;
        const float fv = F == FMT_F16 ? exp2f(-P_SHIFT) : 1.f, fk = scale * exp2f(-shift);
        for (int c = part; c < 2 * HD / 32; c += L::PARTS) {
          const bool is_v = c < HD / 32;
          const int col = 32 * (is_v ? c : c - HD / 32);
          store_row<32, F>((is_v ? t_dv : t_dk) + lane_off + col, is_v ? fv : fk, (is_v ? dst_v : dst_k) + col, row < seq,
                           row < it.n);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(mapa_shared(smem_u32(acc_empty), 0));
      ++ui;
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA leaves while the pair MMAs or remote arrives may touch it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, TMEM_COLS);
  }
}

// ------------------------------------------------------------------ dQ

// The same pair of CTAs with 256 queries: S = Q K^T and dP = dO V^T per key block, dS = P (dP - delta)
// written over S as 16-bit pairs (an A operand in TMEM), dQ += dS K.  S is double-buffered, and dP is
// free as soon as it has been read into registers, so the products of block j + 1 run beside the
// elementwise step of block j.  TMEM: S0 | S1 | dP | dQ.  Thread = query row and a quarter of the keys: lse
// and delta are per thread.  K comes in both cuts, V in rows; three slots each.
struct DqMaps {
  CUtensorMap q, dout, k_rows, k_cols, v_rows, tk_rows, tk_cols;
};

template <int HD>
using DqLayout = Layout<HD, T, 3>;

template <int HD, int F>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(DqLayout<HD>::THREADS, 1)
    bwd_dq_kernel(const __grid_constant__ DqMaps tm, const float* __restrict__ lse2, const float* __restrict__ delta,
                  const float2* __restrict__ norms2, OutRows dq, int batch, int seq, int n_heads,
                  const int32_t* __restrict__ key_lens, const KernelGuard guard) {
  using L = DqLayout<HD>;
  constexpr int N = L::N;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem + L::OFF_A;
  uint8_t* sDO = smem + L::OFF_B;
  uint8_t* sKr = smem + L::OFF_RING;
  uint8_t* sVr = sKr + N * L::CUT;
  uint8_t* sKc = sVr + N * L::CUT;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  const Ring<N> kr(bars), vr(bars + 2 * N), kc(bars + 4 * N);
  const Ring<1> qt(bars + 6 * N), dt(bars + 6 * N + 2);
  uint64_t* s_full = bars + 6 * N + 4;  // [2]
  uint64_t* dp_full = s_full + 2;
  uint64_t* dp_empty = dp_full + 1;     // leader: every elementwise warp of both CTAs
  // leader: every elementwise warp of both CTAs; one per S buffer, since a warp may be done with block u + 1 (whose
  // products do not wait for dS(u)) before another has written its dS(u)
  uint64_t* ds_full = dp_empty + 1;     // [2]
  uint64_t* acc_full = ds_full + 2;
  uint64_t* acc_empty = acc_full + 1;   // leader: every elementwise warp of both CTAs
  uint64_t* drain_bar = acc_empty + 1;
  static_assert(6 * N + 4 + 9 <= L::NUM_BARS, "barriers fit");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + L::OFF_MISC + 4);

  const int warp = static_cast<int>(warp_id());
  const int lane = static_cast<int>(lane_id());
  const int rank = static_cast<int>(cluster_ctarank());
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int nblk = blocks_of(seq) + 1;
  const int ntile = (seq + 2 * T - 1) / (2 * T);
  const int items = batch * n_heads * ntile;

  if (threadIdx.x == 0) {
    kr.init();
    vr.init();
    kc.init();
    qt.init();
    dt.init();
    mbar_init(&s_full[0], 1);
    mbar_init(&s_full[1], 1);
    mbar_init(dp_full, 1);
    mbar_init(dp_empty, 2 * L::EW_WARPS);
    mbar_init(&ds_full[0], 2 * L::EW_WARPS);
    mbar_init(&ds_full[1], 2 * L::EW_WARPS);
    mbar_init(acc_full, 1);
    mbar_init(acc_empty, 2 * L::EW_WARPS);
    mbar_init(drain_bar, 1);
    *abort_flag = 0u;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc_pair(tmem_slot, TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t t_dp = tmem + 256, t_dq = tmem + 384;
  pdl_wait_then_release();

  if (warp == 0) {
    const bool one = elect_one();
    int u = 0, ui = 0;
    int n_kr = 0, n_vr = 0, n_kc = 0, n_q = 0, n_d = 0;
    bool ok = true;
    auto where = [&](int i) { return where_code(ERR_TIMEOUT_ABWD_PRODUCER, rank, i); };
    for (int i = pair; i < items && ok; i += pairs) {
      const Item it = item_of(i, ntile, n_heads, seq, key_lens, T);
      if (it.nb == 0) continue;
      const bool tail = has_tail(it.n, seq, T);
      const int x = it.head * HD, row0 = it.tt * 2 * T + rank * T;
      ok = qt.wait_empty(ui, guard, abort_flag, where(0xFFFF));
      if (!ok) break;
      if (one) load_tile<L, HD>(sQ, &tm.q, qt.arm(ui, leader, 2 * L::TILE), x, row0, it.b);
      ++n_q;
      __syncwarp();
      for (int j = 0; j < it.nb; ++j, ++u) {
        const bool tl = tail && j == it.nb - 1;
        const int st = u % N;
        ok = kr.wait_empty(u, guard, abort_flag, where(u));
        if (!ok) break;
        if (one)
          load_rows_cut<L, HD>(sKr + st * L::CUT, tl ? &tm.tk_rows : &tm.k_rows, kr.arm(u, leader, 2 * L::CUT), x,
                            tl ? 0 : j * T, it.b, rank);
        ++n_kr;
        __syncwarp();
        if (j == 0) {
          ok = dt.wait_empty(ui, guard, abort_flag, where(0xFFFE));
          if (!ok) break;
          if (one) load_tile<L, HD>(sDO, &tm.dout, dt.arm(ui, leader, 2 * L::TILE), x, row0, it.b);
          ++n_d;
          __syncwarp();
        }
        ok = vr.wait_empty(u, guard, abort_flag, where(u));
        if (!ok) break;
        if (one)
          load_rows_cut<L, HD>(sVr + st * L::CUT, &tm.v_rows, vr.arm(u, leader, 2 * L::CUT), x, j * T, it.b, rank);
        ++n_vr;
        __syncwarp();
        ok = kc.wait_empty(u, guard, abort_flag, where(u));
        if (!ok) break;
        if (one)
          load_cols_cut<HD>(sKc + st * L::CUT, tl ? &tm.tk_cols : &tm.k_cols, kc.arm(u, leader, 2 * L::CUT), x,
                            tl ? 0 : j * T, it.b, rank);
        ++n_kc;
        __syncwarp();
      }
      ++ui;
    }
    if (leader) {
      const uint32_t wd = where_code(ERR_TIMEOUT_ABWD_DRAIN, 2, 0);
      qt.drain(n_q, guard, abort_flag, wd);
      dt.drain(n_d, guard, abort_flag, wd);
      kr.drain(n_kr, guard, abort_flag, wd);
      vr.drain(n_vr, guard, abort_flag, wd);
      kc.drain(n_kc, guard, abort_flag, wd);
    }
  } else if (warp == 1) {
    const bool one = elect_one();
    if (leader) {
      auto where = [&](int k, int i) { return where_code(ERR_TIMEOUT_ABWD_MMA, k, i); };
      auto issue_s = [&](int u) {
        mma_rows<L, HD, F>(tmem + 128 * (u & 1), sQ, sKr + (u % N) * L::CUT);
        mma_commit_pair(&s_full[u & 1], 0x3);
        mma_commit_pair(&kr.empty[u % N], 0x3);
      };
      auto issue_dp = [&](int u) {
        mma_rows<L, HD, F>(t_dp, sDO, sVr + (u % N) * L::CUT);
        mma_commit_pair(dp_full, 0x3);
        mma_commit_pair(&vr.empty[u % N], 0x3);
      };
      // block u: S into the buffer whose dS(u - 2) was read by dQ(u - 2), issued before; dP once
      // dP(u - 1) has been read
      auto issue_block = [&](int u, bool last) {
        if (!kr.wait_full(u, guard, abort_flag, where(0, u))) return false;
        tc_fence_after();
        if (one) {
          issue_s(u);
          if (last) mma_commit_pair(&qt.empty[0], 0x3);
        }
        __syncwarp();
        if (!vr.wait_full(u, guard, abort_flag, where(1, u)) ||
            (u > 0 && !mbar_wait(dp_empty, static_cast<uint32_t>(u - 1) & 1u, guard, abort_flag, where(2, u))))
          return false;
        tc_fence_after();
        if (one) {
          issue_dp(u);
          if (last) mma_commit_pair(&dt.empty[0], 0x3);
        }
        __syncwarp();
        return true;
      };
      bool ok = true;
      int u = 0, ui = 0;
      for (int i = pair; i < items && ok; i += pairs) {
        const int nb = item_of(i, ntile, n_heads, seq, key_lens, T).nb;
        if (nb == 0) continue;
        ok = qt.wait_full(ui, guard, abort_flag, where(3, u)) && dt.wait_full(ui, guard, abort_flag, where(4, u)) &&
             issue_block(u, nb == 1);
        for (int j = 0; j < nb && ok; ++j, ++u) {
          if (j + 1 < nb) ok = issue_block(u + 1, j + 2 == nb);
          // the first dQ of an item overwrites an accumulator that both CTAs must have read
          ok = ok && kc.wait_full(u, guard, abort_flag, where(5, u)) &&
               mbar_wait(&ds_full[u & 1], static_cast<uint32_t>(u >> 1) & 1u, guard, abort_flag, where(6, u)) &&
               (j > 0 || ui == 0 ||
                mbar_wait(acc_empty, static_cast<uint32_t>(ui - 1) & 1u, guard, abort_flag, where(7, u)));
          if (!ok) break;
          tc_fence_after();
          if (one) {
            mma_cols<T, HD, F>(t_dq, tmem + 128 * (u & 1), COLS, sKc + (u % N) * L::CUT, j > 0);
            mma_commit_pair(&kc.empty[u % N], 0x3);
          }
          __syncwarp();
        }
        if (ok && one) mma_commit_pair(acc_full, 0x3);
        __syncwarp();
        ++ui;
      }
      if (one) mma_commit_pair(drain_bar, 0x3);
      __syncwarp();
    }
    mbar_wait(drain_bar, 0u, guard, abort_flag, where_code(ERR_TIMEOUT_ABWD_DRAIN, 3, rank), true);
  } else {
    const int part = (warp - 2) >> 2;
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t dp_col = t_dp + lane_off + COLS * part;
    const float scale = HD == 128 ? 0.08838834764831845f : 0.125f;
    const float2 c2 = make_float2(scale * LOG2E, scale * LOG2E);
    auto where = [&](int k, int i) { return where_code(ERR_TIMEOUT_ABWD_SOFTMAX, k, i); };
    bool ok = true;
    int u = 0, ui = 0;
    for (int i = pair; i < items && ok; i += pairs) {
      const Item it = item_of(i, ntile, n_heads, seq, key_lens, T);
      const int row0 = it.tt * 2 * T + rank * T;
      if (it.nb == 0) {
        zero_rows<HD, 32 * L::EW_WARPS>(dq.p + static_cast<int64_t>(it.b) * seq * dq.ld + it.head * HD, dq.ld, row0, seq,
                                        static_cast<int>(threadIdx.x) - 64);
        continue;
      }
      // the padded row vectors reach past the pair's 256 rows
      const int64_t at = it.bh * nblk * T + row0 + r;
      const float l2 = lse2[at];
      const float dl = delta[at];
      const float shift = ds_shift<F>(norms2 + it.bh * nblk, blocks_of(it.n));
      const float tau = F == FMT_F16 ? exp2f(shift - P_SHIFT) : 1.f;
      const float2 nl2 = make_float2(-l2, -l2);
      // tau (dP - delta): one fma on the pair
      const float2 tau2 = make_float2(tau, tau), nd2 = make_float2(-dl * tau, -dl * tau);
      for (int j = 0; j < it.nb; ++j, ++u) {
        const uint32_t s_col = tmem + 128 * (u & 1) + lane_off + COLS * part;
        ok = mbar_wait(&s_full[u & 1], static_cast<uint32_t>(u >> 1) & 1u, guard, abort_flag, where(5, u));
        if (!ok) break;
        tc_fence_after();
        float p[COLS];
        get_part(s_col, p);
#pragma unroll
        for (int k = 0; k < COLS; k += 2) {
          const float2 x = fma2(make_float2(p[k], p[k + 1]), c2, nl2);
          p[k] = ex2_approx(x.x);
          p[k + 1] = ex2_approx(x.y);
        }
        ok = mbar_wait(dp_full, static_cast<uint32_t>(u) & 1u, guard, abort_flag, where(6, u));
        if (!ok) break;
        tc_fence_after();
        float x[COLS];
        get_part(dp_col, x);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(mapa_shared(smem_u32(dp_empty), 0));
#pragma unroll
        for (int k = 0; k < COLS; k += 2) {
          float2 y = F == FMT_F16 ? fma2(make_float2(x[k], x[k + 1]), tau2, nd2) : add2(make_float2(x[k], x[k + 1]), nd2);
          y = mul2(y, make_float2(p[k], p[k + 1]));
          x[k] = y.x;
          x[k + 1] = y.y;
        }
        const int valid = it.n - j * T - COLS * part;  // keys past the tokens: dS = 0 whatever S and dP hold
        if (valid < COLS) {
#pragma unroll
          for (int k = 0; k < COLS; ++k) x[k] = k < valid ? x[k] : 0.f;
        }
        put_part<F>(s_col, x);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(mapa_shared(smem_u32(&ds_full[u & 1]), 0));
      }
      if (!ok) break;
      ok = mbar_wait(acc_full, static_cast<uint32_t>(ui) & 1u, guard, abort_flag, where(7, u));
      if (!ok) break;
      tc_fence_after();
      const int row = row0 + r;
      if (part < HD / 32)
        store_row<32, F>(t_dq + lane_off + 32 * part, scale * exp2f(-shift),
                         dq.p + (static_cast<int64_t>(it.b) * seq + row) * dq.ld + it.head * HD + 32 * part, row < seq,
                         row < it.n);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(mapa_shared(smem_u32(acc_empty), 0));
      ++ui;
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, TMEM_COLS);
  }
}

// ------------------------------------------------------------------ launch

static bool map_rows(CUtensorMap* m, int fmt, const void* p, int64_t ld, int rows, int batch, int cols, int box_cols,
                     int box_rows) {
  const uint64_t dims[3] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(rows), static_cast<uint64_t>(batch)};
  const uint64_t strides[2] = {static_cast<uint64_t>(ld) * 2, static_cast<uint64_t>(rows) * ld * 2};
  const uint32_t box[3] = {static_cast<uint32_t>(box_cols), static_cast<uint32_t>(box_rows), 1};
  return make_tmap(m, fmt == FMT_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                   const_cast<void*>(p), dims, strides, box,
                   box_cols == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
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
  DqMaps mq;
  tile(&mq.q, q);
  tile(&mq.dout, go);
  cuts(&mq.k_rows, &mq.k_cols, k, seq, T);
  cuts(&mq.v_rows, nullptr, v, seq, T);
  cuts(&mq.tk_rows, &mq.tk_cols, tk, T, T);
  DkvMaps mk;
  tile(&mk.k, k);
  tile(&mk.v, v);
  cuts(&mk.q_rows, &mk.q_cols, q, seq, BQ);
  cuts(&mk.do_rows, &mk.do_cols, go, seq, BQ);
  cuts(&mk.tq_rows, &mk.tq_cols, tq, T, BQ);
  cuts(&mk.tdo_rows, &mk.tdo_cols, tdo, T, BQ);
  if (!ok) return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(bwd_dkv_kernel<HD, F>, cudaFuncAttributeMaxDynamicSharedMemorySize, LK::SMEM);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(bwd_dq_kernel<HD, F>, cudaFuncAttributeMaxDynamicSharedMemorySize, LQ::SMEM);
  if (e != cudaSuccess) return e;
  const PrepArgs pa{static_cast<const uint16_t*>(q.p), static_cast<const uint16_t*>(k.p),
                    static_cast<const uint16_t*>(v.p), static_cast<const uint16_t*>(out),
                    static_cast<const uint16_t*>(dout), q.ld, k.ld, v.ld, lse, key_lens, w.lse2, w.delta, w.norms2,
                    w.tails, batch, seq, n_heads};
  e = launch_pdl(bwd_prep_kernel<HD, F>, dim3(nblk, n_heads, batch), dim3(256), 0, s, pa);
  if (e != cudaSuccess) return e;
  int sms = 0, dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    sms = 148;
  const int64_t items = static_cast<int64_t>((seq + 2 * T - 1) / (2 * T)) * n_heads * batch;
  const dim3 grid(2u * static_cast<unsigned>(items < sms / 2 ? items : sms / 2));
  auto view = [](Rows r) { return OutRows{static_cast<uint16_t*>(const_cast<void*>(r.p)), r.ld}; };
  e = launch_pdl(bwd_dq_kernel<HD, F>, grid, dim3(LQ::THREADS), LQ::SMEM, s, mq, w.lse2, w.delta, w.norms2, view(dq), batch,
                 seq, n_heads, key_lens, g);
  if (e != cudaSuccess) return e;
  return launch_pdl(bwd_dkv_kernel<HD, F>, grid, dim3(LK::THREADS), LK::SMEM, s, mk, w.lse2, w.delta, w.norms2, view(dk),
                    view(dv), batch, seq, n_heads, key_lens, g);
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
