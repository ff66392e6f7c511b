// The gradient of the joint attention (Ideogram 4 deep dive, section 4-2: one sequence, one
// bidirectional self-attention), the probabilities recomputed from q, k and the row log-sum-exps:
//   P = exp(q k^T / sqrt(hd) - lse)         delta_q = sum_c dO_qc O_qc
//   dV = P^T dO     dP = dO V^T     dS = P o (dP - delta) / sqrt(hd)     dQ = dS K     dK = dS^T Q
// Three launches:
//   bwd_prep_kernel  delta and the row log-sum-exps in log2 units, padded to whole blocks of 128
//                    rows, and what the other two need to know of the data (see below)
//   bwd_dq_kernel    one query tile per CTA, over all key blocks
//   bwd_dkv_kernel   one key tile per CTA, over all query blocks
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
#include "train.h"

namespace jab {
namespace abwd {

constexpr int T = 128;  // rows of a tile (queries and keys)
constexpr int THREADS = 320;
constexpr int TMEM_COLS = 512;
constexpr int STAGES = 2;
constexpr float LOG2E = 1.4426950408889634f;
constexpr float P_SHIFT = 15.f;  // f16: P is held as 2^15 P

__host__ __device__ inline int blocks_of(int seq) { return (seq + T - 1) / T; }

// Per (b, h), rows padded to whole blocks: ws.lse2 / ws.delta [B, H, nblk * 128]; norms2
// [B, H, nblk]: the block's max |dO_q|^2 and max |V_k|^2 (f16 only); tails: zero-padded copies
// [3: q, k, dO][B, 128, H hd].
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
  const size_t bh = static_cast<size_t>(batch) * n_heads, nblk = blocks_of(seq);
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
// The element's last block is read from its tail copy.
__device__ __forceinline__ bool has_tail(int n, int seq) { return n < seq && n % T != 0; }

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
  if (has_tail(n, a.seq) && blk == n / T) {
    const size_t one = static_cast<size_t>(a.batch) * T * d;
    for (int p = 0; p < PASSES; ++p) {
      const int r = p * ROWS + r0;
      const int row = blk * T + r;
      const int64_t at = static_cast<int64_t>(b) * a.seq + row;
      uint4 x = make_uint4(0u, 0u, 0u, 0u), y = x, z = x;
      if (row < n) {
        x = reinterpret_cast<const uint4*>(a.q + at * a.ldq + h * HD)[c];
        y = reinterpret_cast<const uint4*>(a.k + at * a.ldk + h * HD)[c];
        z = reinterpret_cast<const uint4*>(a.dout + at * d + h * HD)[c];
      }
      uint16_t* dst = a.tails + (static_cast<size_t>(b) * T + r) * d + h * HD;
      reinterpret_cast<uint4*>(dst)[c] = x;
      reinterpret_cast<uint4*>(dst + one)[c] = y;
      reinterpret_cast<uint4*>(dst + 2 * one)[c] = z;
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

template <int HD>
struct Layout {
  static constexpr int SLAB = T * 128;  // 128 rows of 64 values, 128-byte swizzle
  static constexpr int TILE = (HD / 64) * SLAB;
  static constexpr int OFF_A = 0;                       // own tile: K (dkv) / Q (dq)
  static constexpr int OFF_B = OFF_A + TILE;            // own tile: V (dkv) / dO (dq)
  static constexpr int OFF_X = OFF_B + TILE;            // ring: Q (dkv) / K (dq)
  static constexpr int OFF_Y = OFF_X + STAGES * TILE;   // ring: dO (dkv) / V (dq)
  static constexpr int OFF_VEC = OFF_Y + STAGES * TILE;  // ring (dkv): lse2, delta of the block
  static constexpr int OFF_BAR = OFF_VEC + STAGES * 2 * T * 4;
  static constexpr int NUM_BARS = 1 + 4 * STAGES + 8;
  static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;
  static constexpr int SMEM = OFF_MISC + 16 + 1024;
  static_assert(SMEM <= 232448, "227 KB of shared memory per CTA");
};

// Global -> shared copy of a multiple of 16 bytes, both addresses 16-byte aligned.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// One tile of 128 rows x HD at (column x, row y, element z).
template <int HD>
__device__ __forceinline__ void load_tile(uint8_t* dst, const CUtensorMap* m, uint64_t* bar, int x, int y, int z) {
  for (int c = 0; c < HD / 64; ++c) tma_load_3d(dst + c * Layout<HD>::SLAB, m, bar, x + 64 * c, y, z);
}

// D[128 x 128] = A B^T over HD, both tiles 128 rows x HD in shared memory.
template <int HD, int F>
__device__ __forceinline__ void mma_rows(uint32_t d, const uint8_t* a, const uint8_t* b) {
  constexpr uint32_t idesc = idesc_f16kind(T, T, F == FMT_F16, false, false);
  const uint32_t ab = smem_u32(a), bb = smem_u32(b);
#pragma unroll
  for (int kk = 0; kk < HD / 16; ++kk) {
    const uint32_t off = (kk >> 2) * Layout<HD>::SLAB + (kk & 3) * 32;
    mma_f16kind_ss(d, smem_desc_sw128(ab + off, 16, 1024), smem_desc_sw128(bb + off, 16, 1024), idesc, kk > 0 ? 1u : 0u);
  }
}

// D[128 x HD] (+)= A[128 x 128] B, A as 16-bit pairs in TMEM (its k-th half of 64 columns at
// a + 64 k, see put_half), B a tile of 128 rows x HD in shared memory read with its rows as the
// contraction axis (slabs of 64 columns, one leading-dimension step apart).
template <int HD, int F>
__device__ __forceinline__ void mma_cols(uint32_t d, uint32_t a, const uint8_t* b, bool accumulate) {
  constexpr uint32_t idesc = idesc_f16kind(T, HD, F == FMT_F16, false, true);
  const uint32_t bb = smem_u32(b);
#pragma unroll
  for (int kk = 0; kk < T / 16; ++kk)
    mma_f16kind_ts(d, a + 64 * (kk >> 2) + 8 * (kk & 3), smem_desc_sw128(bb + kk * 16 * 128, Layout<HD>::SLAB, 1024),
                   idesc, (accumulate || kk > 0) ? 1u : 0u);
}

__device__ __forceinline__ void get_half(uint32_t taddr, float (&v)[64]) {
  uint32_t a[32], b[32];
  tmem_ld32(taddr, a);
  tmem_ld32(taddr + 32, b);
  tmem_ld_wait_regs(a);
  tmem_ld_wait_regs(b);
#pragma unroll
  for (int k = 0; k < 32; ++k) {
    v[k] = __uint_as_float(a[k]);
    v[32 + k] = __uint_as_float(b[k]);
  }
}

// 64 values as 16-bit pairs into the first 32 of the 64 columns that they came from.
template <int F>
__device__ __forceinline__ void put_half(uint32_t taddr, const float (&v)[64]) {
  uint32_t pk[32];
#pragma unroll
  for (int k = 0; k < 32; ++k) pk[k] = pack2<F>(v[2 * k], v[2 * k + 1]);
  tmem_st32(taddr, pk);
  tmem_st_wait();
}

// One accumulator row (HD fp32 columns at taddr) times f into a 16-bit row, or zeros.
template <int HD, int F>
__device__ __forceinline__ void store_row(uint32_t taddr, float f, uint16_t* dst, bool in_range, bool live) {
#pragma unroll
  for (int c = 0; c < HD / 32; ++c) {
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

// Zeros into the rows [row0, row0 + 128) below seq of one head (the whole CTA calls it).
template <int HD>
__device__ __forceinline__ void zero_rows(uint16_t* base, int64_t ld, int row0, int seq) {
  constexpr int LANES = HD / 8;
  for (int i = threadIdx.x; i < T * LANES; i += THREADS) {
    const int row = row0 + i / LANES;
    if (row < seq) reinterpret_cast<uint4*>(base + row * ld)[i % LANES] = make_uint4(0u, 0u, 0u, 0u);
  }
}

struct OutRows {
  uint16_t* p;
  int64_t ld;
};

// ------------------------------------------------------------------ dK, dV

// One key tile per CTA.  The products run with the keys as rows (S^T = K Q^T, dP^T = V dO^T), so
// that P^T and dS^T come out of the elementwise step in the very layout in which the tensor core
// reads an A operand from TMEM: dV += P^T dO, dK += dS^T Q.  TMEM: S^T | dP^T | dV | dK, 128 columns
// each; P^T and dS^T overwrite S^T and dP^T as 16-bit pairs.
//   warp 0       loads: K and V of the tile, then per query block Q, dO and their row vectors
//   warp 1       TMEM; one lane issues  dV(j), S(j+1)  when P(j) is written, and
//                dK(j), dP(j+1)  when dS(j) is, so that each elementwise step runs beside the two
//                products that do not need it
//   warps 2..9   P^T = exp2(c S^T - lse2), then dS^T = P^T (dP^T - delta); thread = key row and
//                half of the query columns.
template <int HD, int F>
__global__ void __launch_bounds__(THREADS, 1)
    bwd_dkv_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                   const __grid_constant__ CUtensorMap tm_qt, const __grid_constant__ CUtensorMap tm_dot,
                   const float* __restrict__ lse2, const float* __restrict__ delta, const float2* __restrict__ norms2,
                   OutRows dk, OutRows dv, int seq, int n_heads, const int32_t* __restrict__ key_lens,
                   const KernelGuard guard) {
  using L = Layout<HD>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sK = smem + L::OFF_A;
  uint8_t* sV = smem + L::OFF_B;
  uint8_t* sQ = smem + L::OFF_X;
  uint8_t* sDO = smem + L::OFF_Y;
  float* sVec = reinterpret_cast<float*>(smem + L::OFF_VEC);  // [STAGES][lse2 128 | delta 128]
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  uint64_t* kv_full = bars;
  uint64_t* q_full = kv_full + 1;         // [STAGES]
  uint64_t* do_full = q_full + STAGES;    // [STAGES]
  uint64_t* empty = do_full + STAGES;     // [STAGES] every product of the block is done
  uint64_t* s_full = empty + STAGES;
  uint64_t* dp_full = s_full + 1;
  uint64_t* p_full = dp_full + 1;         // 8 warps
  uint64_t* ds_full = p_full + 1;         // 8 warps
  uint64_t* acc_full = ds_full + 1;       // dV, dK final (and every MMA retired)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + L::OFF_MISC + 4);

  const int warp = static_cast<int>(warp_id());
  const int lane = static_cast<int>(lane_id());
  const int nblk = blocks_of(seq);
  const int kt = static_cast<int>(blockIdx.x % nblk);
  const int64_t bh = blockIdx.x / nblk;
  const int head = static_cast<int>(bh % n_heads);
  const int b = static_cast<int>(bh / n_heads);

  if (threadIdx.x == 0) {
    mbar_init(kv_full, 1);
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&do_full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(s_full, 1);
    mbar_init(dp_full, 1);
    mbar_init(p_full, 8);
    mbar_init(ds_full, 8);
    mbar_init(acc_full, 1);
    *abort_flag = 0u;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc(tmem_slot, TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t t_s = tmem, t_dp = tmem + 128, t_dv = tmem + 256, t_dk = tmem + 384;
  pdl_wait_then_release();

  const int n = tokens_of(key_lens, b, seq);
  const int nb = kt * T < n ? blocks_of(n) : 0;  // a tile past the tokens has nothing to add up
  const bool tail = has_tail(n, seq);
  uint16_t* dk_head = dk.p + static_cast<int64_t>(b) * seq * dk.ld + head * HD;
  uint16_t* dv_head = dv.p + static_cast<int64_t>(b) * seq * dv.ld + head * HD;

  if (nb == 0) {
    zero_rows<HD>(dk_head, dk.ld, kt * T, seq);
    zero_rows<HD>(dv_head, dv.ld, kt * T, seq);
  } else if (warp == 0) {
    if (lane == 0) {
      mbar_arrive_expect_tx(kv_full, 2 * L::TILE);
      load_tile<HD>(sK, &tm_k, kv_full, head * HD, kt * T, b);
      load_tile<HD>(sV, &tm_v, kv_full, head * HD, kt * T, b);
    }
    __syncwarp();
    int issued = 0;
    for (int j = 0; j < nb; ++j) {
      const int st = j % STAGES;
      if (!mbar_wait(&empty[st], (static_cast<uint32_t>(j / STAGES) & 1u) ^ 1u, guard, abort_flag,
                     where_code(ERR_TIMEOUT_ABWD_PRODUCER, 0, j)))
        break;
      if (lane == 0) {
        const bool from_tail = tail && j == nb - 1;
        const CUtensorMap* mq = from_tail ? &tm_qt : &tm_q;
        const CUtensorMap* mo = from_tail ? &tm_dot : &tm_do;
        const int y = from_tail ? 0 : j * T;
        float* vec = sVec + st * 2 * T;
        mbar_arrive_expect_tx(&q_full[st], L::TILE + T * 4);
        load_tile<HD>(sQ + st * L::TILE, mq, &q_full[st], head * HD, y, b);
        bulk_load(vec, lse2 + (bh * nblk + j) * T, T * 4, &q_full[st]);
        mbar_arrive_expect_tx(&do_full[st], L::TILE + T * 4);
        load_tile<HD>(sDO + st * L::TILE, mo, &do_full[st], head * HD, y, b);
        bulk_load(vec + T, delta + (bh * nblk + j) * T, T * 4, &do_full[st]);
      }
      __syncwarp();
      ++issued;
    }
    // never leave with copies in flight
    mbar_wait(kv_full, 0u, guard, abort_flag, where_code(ERR_TIMEOUT_ABWD_DRAIN, 0, 0), true);
    for (int st = 0; st < STAGES && st < issued; ++st) {
      const uint32_t par = static_cast<uint32_t>((issued - 1 - st) / STAGES) & 1u;
      mbar_wait(&q_full[st], par, guard, abort_flag, where_code(ERR_TIMEOUT_ABWD_DRAIN, 0, st), true);
      mbar_wait(&do_full[st], par, guard, abort_flag, where_code(ERR_TIMEOUT_ABWD_DRAIN, 0, st), true);
    }
  } else if (warp == 1) {
    auto full = [&](uint64_t* ring, int j) {
      return mbar_wait(&ring[j % STAGES], static_cast<uint32_t>(j / STAGES) & 1u, guard, abort_flag,
                       where_code(ERR_TIMEOUT_ABWD_MMA, 0, j));
    };
    auto issue_s = [&](int j) {
      mma_rows<HD, F>(t_s, sK, sQ + (j % STAGES) * L::TILE);
      mma_commit(s_full);
    };
    auto issue_dp = [&](int j) {
      mma_rows<HD, F>(t_dp, sV, sDO + (j % STAGES) * L::TILE);
      mma_commit(dp_full);
    };
    bool ok = mbar_wait(kv_full, 0u, guard, abort_flag, where_code(ERR_TIMEOUT_ABWD_MMA, 1, 0)) && full(q_full, 0) &&
              full(do_full, 0);
    if (ok) {
      tc_fence_after();
      if (lane == 0) {
        issue_s(0);
        issue_dp(0);
      }
      __syncwarp();
    }
    for (int j = 0; j < nb && ok; ++j) {
      const bool next = j + 1 < nb;
      const uint32_t par = static_cast<uint32_t>(j) & 1u;
      ok = mbar_wait(p_full, par, guard, abort_flag, where_code(ERR_TIMEOUT_ABWD_MMA, 2, j)) &&
           (!next || full(q_full, j + 1));
      if (!ok) break;
      tc_fence_after();
      if (lane == 0) {
        mma_cols<HD, F>(t_dv, t_s, sDO + (j % STAGES) * L::TILE, j > 0);
        if (next) issue_s(j + 1);  // overwrites P(j) only after dV(j) has read it (in-order issue)
      }
      __syncwarp();
      ok = mbar_wait(ds_full, par, guard, abort_flag, where_code(ERR_TIMEOUT_ABWD_MMA, 3, j)) &&
           (!next || full(do_full, j + 1));
      if (!ok) break;
      tc_fence_after();
      if (lane == 0) {
        mma_cols<HD, F>(t_dk, t_dp, sQ + (j % STAGES) * L::TILE, j > 0);
        mma_commit(&empty[j % STAGES]);
        if (next) issue_dp(j + 1);
      }
      __syncwarp();
    }
    if (lane == 0) mma_commit(acc_full);
    __syncwarp();
    mbar_wait(acc_full, 0u, guard, abort_flag, where_code(ERR_TIMEOUT_ABWD_DRAIN, 1, 0), true);
  } else {
    const int half = (warp - 2) >> 2;
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t s_col = t_s + lane_off + 64 * half;
    const uint32_t dp_col = t_dp + lane_off + 64 * half;
    const float scale = HD == 128 ? 0.08838834764831845f : 0.125f;
    const float shift = ds_shift<F>(norms2 + bh * nblk, blocks_of(n));
    // P carries 2^15 in f16; dS = that P times (dP - delta) times tau = 2^(shift - 15)
    const float tau = F == FMT_F16 ? exp2f(shift - P_SHIFT) : 1.f;
    const float2 c2 = make_float2(scale * LOG2E, scale * LOG2E);
    bool ok = true;
    for (int j = 0; j < nb; ++j) {
      const uint32_t par = static_cast<uint32_t>(j) & 1u;
      const float* vec = sVec + (j % STAGES) * 2 * T + 64 * half;
      // the row vectors ride on the ring's own barriers
      ok = mbar_wait(&q_full[j % STAGES], static_cast<uint32_t>(j / STAGES) & 1u, guard, abort_flag,
                     where_code(ERR_TIMEOUT_ABWD_SOFTMAX, 0, j)) &&
           mbar_wait(s_full, par, guard, abort_flag, where_code(ERR_TIMEOUT_ABWD_SOFTMAX, 1, j));
      if (!ok) break;
      tc_fence_after();
      float p[64];
      get_half(s_col, p);
#pragma unroll
      for (int k = 0; k < 64; k += 2) {
        const float2 l = *reinterpret_cast<const float2*>(vec + k);
        const float2 x = fma2(make_float2(p[k], p[k + 1]), c2, make_float2(-l.x, -l.y));
        p[k] = ex2_approx(x.x);
        p[k + 1] = ex2_approx(x.y);
      }
      put_half<F>(s_col, p);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full);
      ok = mbar_wait(&do_full[j % STAGES], static_cast<uint32_t>(j / STAGES) & 1u, guard, abort_flag,
                     where_code(ERR_TIMEOUT_ABWD_SOFTMAX, 2, j)) &&
           mbar_wait(dp_full, par, guard, abort_flag, where_code(ERR_TIMEOUT_ABWD_SOFTMAX, 3, j));
      if (!ok) break;
      tc_fence_after();
      float x[64];
      get_half(dp_col, x);
#pragma unroll
      for (int k = 0; k < 64; k += 2) {
        const float2 dl = *reinterpret_cast<const float2*>(vec + T + k);
        float2 y = add2(make_float2(x[k], x[k + 1]), make_float2(-dl.x, -dl.y));
        y = mul2(y, make_float2(p[k], p[k + 1]));
        if constexpr (F == FMT_F16) y = mul2(y, make_float2(tau, tau));
        x[k] = y.x;
        x[k + 1] = y.y;
      }
      put_half<F>(dp_col, x);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(ds_full);
    }
    if (ok && mbar_wait(acc_full, 0u, guard, abort_flag, where_code(ERR_TIMEOUT_ABWD_SOFTMAX, 4, nb))) {
      tc_fence_after();
      const int row = kt * T + r;
      if (half == 0)
        store_row<HD, F>(t_dv + lane_off, F == FMT_F16 ? exp2f(-P_SHIFT) : 1.f, dv_head + row * dv.ld, row < seq,
                         row < n);
      else
        store_row<HD, F>(t_dk + lane_off, scale * exp2f(-shift), dk_head + row * dk.ld, row < seq, row < n);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

// ------------------------------------------------------------------ dQ

// One query tile per CTA: S = Q K^T and dP = dO V^T per key block, dS = P (dP - delta) written over
// S as 16-bit pairs (an A operand in TMEM), dQ += dS K.  S is double-buffered, and dP is free as
// soon as it has been read into registers, so the products of block j + 1 run beside the
// elementwise step of block j.  TMEM: S0 | S1 | dP | dQ.  Thread = query row and half of the keys:
// lse and delta are per thread.
template <int HD, int F>
__global__ void __launch_bounds__(THREADS, 1)
    bwd_dq_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                  const __grid_constant__ CUtensorMap tm_kt, const float* __restrict__ lse2,
                  const float* __restrict__ delta, const float2* __restrict__ norms2, OutRows dq, int seq, int n_heads,
                  const int32_t* __restrict__ key_lens, const KernelGuard guard) {
  using L = Layout<HD>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem + L::OFF_A;
  uint8_t* sDO = smem + L::OFF_B;
  uint8_t* sK = smem + L::OFF_X;
  uint8_t* sV = smem + L::OFF_Y;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  uint64_t* q_full = bars;
  uint64_t* kv_full = q_full + 1;        // [STAGES]
  uint64_t* kv_empty = kv_full + STAGES;  // [STAGES]
  uint64_t* s_full = kv_empty + STAGES;  // [2]
  uint64_t* dp_full = s_full + 2;
  uint64_t* dp_empty = dp_full + 1;      // 8 warps
  uint64_t* ds_full = dp_empty + 1;      // 8 warps
  uint64_t* acc_full = ds_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + L::OFF_MISC + 4);

  const int warp = static_cast<int>(warp_id());
  const int lane = static_cast<int>(lane_id());
  const int nblk = blocks_of(seq);
  const int qt = static_cast<int>(blockIdx.x % nblk);
  const int64_t bh = blockIdx.x / nblk;
  const int head = static_cast<int>(bh % n_heads);
  const int b = static_cast<int>(bh / n_heads);

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 1);
    }
    mbar_init(&s_full[0], 1);
    mbar_init(&s_full[1], 1);
    mbar_init(dp_full, 1);
    mbar_init(dp_empty, 8);
    mbar_init(ds_full, 8);
    mbar_init(acc_full, 1);
    *abort_flag = 0u;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc(tmem_slot, TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t t_dp = tmem + 256, t_dq = tmem + 384;
  pdl_wait_then_release();

  const int n = tokens_of(key_lens, b, seq);
  const int nb = qt * T < n ? blocks_of(n) : 0;
  const bool tail = has_tail(n, seq);
  uint16_t* dq_head = dq.p + static_cast<int64_t>(b) * seq * dq.ld + head * HD;

  if (nb == 0) {
    zero_rows<HD>(dq_head, dq.ld, qt * T, seq);
  } else if (warp == 0) {
    if (lane == 0) {
      mbar_arrive_expect_tx(q_full, 2 * L::TILE);
      load_tile<HD>(sQ, &tm_q, q_full, head * HD, qt * T, b);
      load_tile<HD>(sDO, &tm_do, q_full, head * HD, qt * T, b);
    }
    __syncwarp();
    int issued = 0;
    for (int j = 0; j < nb; ++j) {
      const int st = j % STAGES;
      if (!mbar_wait(&kv_empty[st], (static_cast<uint32_t>(j / STAGES) & 1u) ^ 1u, guard, abort_flag,
                     where_code(ERR_TIMEOUT_ABWD_PRODUCER, 1, j)))
        break;
      if (lane == 0) {
        const bool from_tail = tail && j == nb - 1;
        mbar_arrive_expect_tx(&kv_full[st], 2 * L::TILE);
        load_tile<HD>(sK + st * L::TILE, from_tail ? &tm_kt : &tm_k, &kv_full[st], head * HD, from_tail ? 0 : j * T, b);
        load_tile<HD>(sV + st * L::TILE, &tm_v, &kv_full[st], head * HD, j * T, b);
      }
      __syncwarp();
      ++issued;
    }
    mbar_wait(q_full, 0u, guard, abort_flag, where_code(ERR_TIMEOUT_ABWD_DRAIN, 2, 0), true);
    for (int st = 0; st < STAGES && st < issued; ++st)
      mbar_wait(&kv_full[st], static_cast<uint32_t>((issued - 1 - st) / STAGES) & 1u, guard, abort_flag,
                where_code(ERR_TIMEOUT_ABWD_DRAIN, 2, st), true);
  } else if (warp == 1) {
    auto full = [&](int j) {
      return mbar_wait(&kv_full[j % STAGES], static_cast<uint32_t>(j / STAGES) & 1u, guard, abort_flag,
                       where_code(ERR_TIMEOUT_ABWD_MMA, 4, j));
    };
    auto issue_s = [&](int j) {
      mma_rows<HD, F>(tmem + 128 * (j & 1), sQ, sK + (j % STAGES) * L::TILE);
      mma_commit(&s_full[j & 1]);
    };
    auto issue_dp = [&](int j) {
      mma_rows<HD, F>(t_dp, sDO, sV + (j % STAGES) * L::TILE);
      mma_commit(dp_full);
    };
    bool ok = mbar_wait(q_full, 0u, guard, abort_flag, where_code(ERR_TIMEOUT_ABWD_MMA, 5, 0)) && full(0);
    if (ok) {
      tc_fence_after();
      if (lane == 0) {
        issue_s(0);
        issue_dp(0);
      }
      __syncwarp();
    }
    for (int j = 0; j < nb && ok; ++j) {
      const uint32_t par = static_cast<uint32_t>(j) & 1u;
      if (j + 1 < nb) {
        ok = full(j + 1);
        if (!ok) break;
        tc_fence_after();
        if (lane == 0) issue_s(j + 1);  // into the buffer whose dS(j-1) was read by dQ(j-1), issued before
        __syncwarp();
        ok = mbar_wait(dp_empty, par, guard, abort_flag, where_code(ERR_TIMEOUT_ABWD_MMA, 6, j));
        if (!ok) break;
        tc_fence_after();
        if (lane == 0) issue_dp(j + 1);
        __syncwarp();
      }
      ok = mbar_wait(ds_full, par, guard, abort_flag, where_code(ERR_TIMEOUT_ABWD_MMA, 7, j));
      if (!ok) break;
      tc_fence_after();
      if (lane == 0) {
        mma_cols<HD, F>(t_dq, tmem + 128 * (j & 1), sK + (j % STAGES) * L::TILE, j > 0);
        mma_commit(&kv_empty[j % STAGES]);
      }
      __syncwarp();
    }
    if (lane == 0) mma_commit(acc_full);
    __syncwarp();
    mbar_wait(acc_full, 0u, guard, abort_flag, where_code(ERR_TIMEOUT_ABWD_DRAIN, 3, 0), true);
  } else {
    const int half = (warp - 2) >> 2;
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t dp_col = t_dp + lane_off + 64 * half;
    const float scale = HD == 128 ? 0.08838834764831845f : 0.125f;
    const float shift = ds_shift<F>(norms2 + bh * nblk, blocks_of(n));
    const float tau = F == FMT_F16 ? exp2f(shift - P_SHIFT) : 1.f;
    const float l2 = lse2[(bh * nblk + qt) * T + r];
    const float dl = delta[(bh * nblk + qt) * T + r];
    const float2 c2 = make_float2(scale * LOG2E, scale * LOG2E);
    const float2 nl2 = make_float2(-l2, -l2);
    // tau (dP - delta): one fma on the pair
    const float2 tau2 = make_float2(tau, tau), nd2 = make_float2(-dl * tau, -dl * tau);
    bool ok = true;
    for (int j = 0; j < nb; ++j) {
      const uint32_t s_col = tmem + 128 * (j & 1) + lane_off + 64 * half;
      ok = mbar_wait(&s_full[j & 1], static_cast<uint32_t>(j >> 1) & 1u, guard, abort_flag,
                     where_code(ERR_TIMEOUT_ABWD_SOFTMAX, 5, j));
      if (!ok) break;
      tc_fence_after();
      float p[64];
      get_half(s_col, p);
#pragma unroll
      for (int k = 0; k < 64; k += 2) {
        const float2 x = fma2(make_float2(p[k], p[k + 1]), c2, nl2);
        p[k] = ex2_approx(x.x);
        p[k + 1] = ex2_approx(x.y);
      }
      ok = mbar_wait(dp_full, static_cast<uint32_t>(j) & 1u, guard, abort_flag,
                     where_code(ERR_TIMEOUT_ABWD_SOFTMAX, 6, j));
      if (!ok) break;
      tc_fence_after();
      float x[64];
      get_half(dp_col, x);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(dp_empty);
#pragma unroll
      for (int k = 0; k < 64; k += 2) {
        float2 y = F == FMT_F16 ? fma2(make_float2(x[k], x[k + 1]), tau2, nd2) : add2(make_float2(x[k], x[k + 1]), nd2);
        y = mul2(y, make_float2(p[k], p[k + 1]));
        x[k] = y.x;
        x[k + 1] = y.y;
      }
      const int valid = n - j * T - 64 * half;  // keys past the tokens: dS = 0 whatever S and dP hold
      if (valid < 64) {
#pragma unroll
        for (int k = 0; k < 64; ++k) x[k] = k < valid ? x[k] : 0.f;
      }
      put_half<F>(s_col, x);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(ds_full);
    }
    if (ok && mbar_wait(acc_full, 0u, guard, abort_flag, where_code(ERR_TIMEOUT_ABWD_SOFTMAX, 7, nb)) && half == 0) {
      tc_fence_after();
      const int row = qt * T + r;
      store_row<HD, F>(t_dq + lane_off, scale * exp2f(-shift), dq_head + row * dq.ld, row < seq, row < n);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

// ------------------------------------------------------------------ launch

static bool map_rows(CUtensorMap* m, int fmt, const void* p, int64_t ld, int rows, int batch, int cols) {
  const uint64_t dims[3] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(rows), static_cast<uint64_t>(batch)};
  const uint64_t strides[2] = {static_cast<uint64_t>(ld) * 2, static_cast<uint64_t>(rows) * ld * 2};
  const uint32_t box[3] = {64, T, 1};
  return make_tmap(m, fmt == FMT_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                   const_cast<void*>(p), dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int HD, int F>
static cudaError_t launch_hd(Rows q, Rows k, Rows v, const void* out, const void* dout, const float* lse, Rows dq,
                             Rows dk, Rows dv, int batch, int seq, int n_heads, const int32_t* key_lens,
                             void* workspace, const KernelGuard& g, cudaStream_t s) {
  using L = Layout<HD>;
  const Workspace w = carve(workspace, batch, seq, n_heads, HD);
  const int d = n_heads * HD, nblk = blocks_of(seq);
  const size_t one = static_cast<size_t>(batch) * T * d;
  CUtensorMap tq, tk, tv, tdo, tqt, tkt, tdot;
  if (!map_rows(&tq, F, q.p, q.ld, seq, batch, d) || !map_rows(&tk, F, k.p, k.ld, seq, batch, d) ||
      !map_rows(&tv, F, v.p, v.ld, seq, batch, d) || !map_rows(&tdo, F, dout, d, seq, batch, d) ||
      !map_rows(&tqt, F, w.tails, d, T, batch, d) || !map_rows(&tkt, F, w.tails + one, d, T, batch, d) ||
      !map_rows(&tdot, F, w.tails + 2 * one, d, T, batch, d))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(bwd_dkv_kernel<HD, F>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(bwd_dq_kernel<HD, F>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM);
  if (e != cudaSuccess) return e;
  const PrepArgs pa{static_cast<const uint16_t*>(q.p), static_cast<const uint16_t*>(k.p),
                    static_cast<const uint16_t*>(v.p), static_cast<const uint16_t*>(out),
                    static_cast<const uint16_t*>(dout), q.ld, k.ld, v.ld, lse, key_lens, w.lse2, w.delta, w.norms2,
                    w.tails, batch, seq, n_heads};
  e = launch_pdl(bwd_prep_kernel<HD, F>, dim3(nblk, n_heads, batch), dim3(256), 0, s, pa);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(nblk) * n_heads * batch));
  auto rows = [](Rows r) { return OutRows{static_cast<uint16_t*>(const_cast<void*>(r.p)), r.ld}; };
  e = launch_pdl(bwd_dq_kernel<HD, F>, grid, dim3(THREADS), L::SMEM, s, tq, tk, tv, tdo, tkt, w.lse2, w.delta,
                 w.norms2, rows(dq), seq, n_heads, key_lens, g);
  if (e != cudaSuccess) return e;
  return launch_pdl(bwd_dkv_kernel<HD, F>, grid, dim3(THREADS), L::SMEM, s, tq, tk, tv, tdo, tqt, tdot, w.lse2,
                    w.delta, w.norms2, rows(dk), rows(dv), seq, n_heads, key_lens, g);
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
