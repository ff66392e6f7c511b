// HBM-bound gradients: QK-RMSNorm + 3D M-RoPE and the row RMSNorm, each with the sums of its
// gains' gradients.  fp32 math.  The sums are taken in a fixed order (registers over a CTA's
// tokens or rows, then shared memory, then one partial row per CTA that a second kernel adds up), so
// a result does not change from run to run.
#include <type_traits>

#include "common.cuh"
#include "pipeline.cuh"
#include "rope.cuh"
#include "train.h"

namespace jab {
namespace tew {

constexpr int SMS = 148;  // grids are multiples of it; the workspaces hold a partial row per CTA

// dst[c] = sum over the n rows of part [n, cols]; one CTA per 32 columns, 32 row lanes each.  Latency-bound:
// 296 rows of 4096 columns (4.8 MB, from L2) 5.7 us, 148 rows of 256 columns 4.9 us.
__global__ void __launch_bounds__(1024) sum_rows_kernel(const float* __restrict__ part, int n, int64_t cols,
                                                        float* __restrict__ dst0, float* __restrict__ dst1,
                                                        int64_t split) {
  __shared__ float red[32][33];
  pdl_wait_then_release();
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int64_t c = blockIdx.x * 32ll + x;
  float acc = 0.f;
  if (c < cols)
    for (int r = y; r < n; r += 32) acc += part[r * cols + c];
  red[y][x] = acc;
  __syncthreads();
  if (y != 0 || c >= cols) return;
  acc = 0.f;
#pragma unroll
  for (int k = 0; k < 32; ++k) acc += red[k][x];
  if (c < split)
    dst0[c] = acc;
  else
    dst1[c - split] = acc;
}

static cudaError_t sum_rows(const float* part, int n, int64_t cols, float* dst0, float* dst1, int64_t split,
                            cudaStream_t s) {
  return launch_pdl(sum_rows_kernel, dim3(static_cast<unsigned>((cols + 31) / 32)), dim3(1024), 0, s, part, n, cols,
                    dst0, dst1, split);
}

constexpr int MAX_STAGES = 8;

// The QK-norm gradient's CTAs per SM: one above 256 threads a token, else what fits with 96 registers a
// thread, of which an SM's four quarters hold five warps each (two CTAs of 256 threads and the two warps of
// angles).  A CTA works on one token at a time, so that
// narrow models need many: event-timed with L2 cold, 4 x 4608 tokens of 4 or 8 heads of 64 54 us (two CTAs
// 118, seven, one of them in a second wave, 70), 2 x 4608 of 16 heads of 64 38 us (63) and of 128 58 us (69).
constexpr int qk_ctas(int per_token) {
  return per_token > 256 ? 1 : 20 / ((per_token + 31) / 32 + 2);
}

// (b, s) of the tokens blockIdx.x, blockIdx.x + gridDim.x, ... without a division for each.
struct TokenWalk {
  int b, s, db, ds;
  __device__ __forceinline__ TokenWalk(int seq)
      : b(blockIdx.x / seq), s(blockIdx.x % seq), db(gridDim.x / seq), ds(gridDim.x % seq) {}
  __device__ __forceinline__ void step(int seq) {
    b += db;
    s += ds;
    if (s >= seq) {
      s -= seq;
      ++b;
    }
  }
};

// ------------------------------------------------------------------ QK-RMSNorm + M-RoPE

// With x a raw head vector, r = (mean x^2 + eps)^(-1/2), xh = r x, u = xh g and y = R u (R the
// token's rotation of the pairs (i, i + hd/2)): dz = R^T dy, dg = sum dz xh, du = dz g and
// dx = r (du - xh mean(du xh)).
// A CTA works on q or on k (blockIdx.y) and walks tokens with the gain's sums in registers (q and k
// together needed more registers than two CTAs of an SM have); thread layout as in the forward kernel,
// one thread per head and 8 rotary pairs.  The last two warps run ahead: they copy a token's raw rows and
// gradients into a ring of shared memory with two bulk copies and compute its angles beside them, an
// angle per lane, so that the other warps wait for neither memory nor fp64.  4608 tokens x 32 heads of 128,
// L2 cold: 52 us event-timed with the sums' kernel (226 MB, 4.4 TB/s); alone 46.6 us with instructions issued
// in 65 % of the cycles, so it is bound by neither memory nor issue alone; with one warp of angles 58 us.
// 16896 tokens 150 us (5.5 TB/s).
// Tokens behind an element's count are not read; their gradients are zeros.
template <int F, int HD, int MAX_THREADS>
__global__ void __launch_bounds__(MAX_THREADS + 64, qk_ctas(MAX_THREADS))
    qknorm_mrope_bwd_kernel(const uint16_t* __restrict__ qkv, const uint16_t* dqk, int64_t ld_dqk, uint16_t* dx,
                            int64_t ld_dx, float* __restrict__ part, int64_t tokens, int seq, int n_heads, RopeArgs ra,
                            const uint16_t* __restrict__ g_q, const uint16_t* __restrict__ g_k, float eps, int stages,
                            const KernelGuard guard) {
  const bool is_k = blockIdx.y != 0;
  constexpr int half = HD / 2;
  constexpr int GROUP = HD / 16;  // threads per head
  __shared__ __align__(16) float s_cos[MAX_STAGES][half], s_sin[MAX_STAGES][half];
  __shared__ uint64_t full[MAX_STAGES], empty[MAX_STAGES];
  __shared__ uint32_t abort_flag;
  extern __shared__ __align__(16) uint8_t ring[];  // [stages][raw | gradient]; at the end [warps][HD] sums
  const int per_token = n_heads * GROUP;
  const int warps = (blockDim.x >> 5) - 2, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int d = n_heads * HD;
  const uint32_t row_bytes = 2u * d;
  const int col = is_k ? d : 0;
  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(&full[i], 2);
      mbar_init(&empty[i], warps);
    }
    abort_flag = 0u;
    fence_barrier_init();
  }
  __syncthreads();
  pdl_wait_then_release();

  if (warp >= warps) {
    const bool first = warp == warps;
    // this lane's pair: its frequency and axis, once for all tokens (read per token, from where the lanes'
    // addresses differ, 16896 tokens of 32 heads of 128 took 155 us against 150)
    const int i = first ? lane : lane + 32;
    const float freq = i < half ? ra.inv_freq[i] : 0.f;
    const int axis = i < ra.sec_t ? 0 : i < ra.sec_t + ra.sec_h ? 1 : 2;
    int u = 0;
    TokenWalk w(seq);
    for (int64_t bs = blockIdx.x; bs < tokens; bs += gridDim.x, w.step(seq)) {
      const int b = w.b, s = w.s;
      if (s >= rope_count(ra, b)) continue;
      int pt, ph, pw;
      rope_position(ra, b, s, pt, ph, pw);
      const int st = u % stages;
      const bool got = mbar_wait(&empty[st], (static_cast<uint32_t>(u / stages) & 1u) ^ 1u, guard, &abort_flag,
                                 where_code(ERR_TIMEOUT_QKBWD, 0, u));
      if (first && lane == 0 && got) {
        // the angles below are part of the phase: its two arrivals come after them
        asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(&full[st])),
                     "r"(2 * row_bytes)
                     : "memory");
        bulk_load(ring + st * 2 * row_bytes, qkv + bs * 3 * d + col, row_bytes, &full[st]);
        bulk_load(ring + st * 2 * row_bytes + row_bytes, dqk + bs * ld_dqk + col, row_bytes, &full[st]);
      }
      if (i < half) rope_angle(freq, axis == 0 ? pt : axis == 1 ? ph : pw, s_cos[st][i], s_sin[st][i]);
      // the lanes' stores come before lane 0's release; the vote below orders no memory
      __syncwarp();
      if (lane == 0 && got) mbar_arrive(&full[st]);
      const bool all = __all_sync(0xffffffffu, got);
      ++u;
      if (!all) break;  // a wait gave up: the warp leaves as a whole
    }
    // never leave with copies in flight
    if (first) {
      for (int v = u > stages ? u - stages : 0; v < u; ++v)
        mbar_wait(&full[v % stages], static_cast<uint32_t>(v / stages) & 1u, guard, &abort_flag,
                  where_code(ERR_TIMEOUT_QKBWD, 1, v), true);
    }
    __syncthreads();
    __syncthreads();
    return;
  }

  const bool mine = static_cast<int>(threadIdx.x) < per_token;
  const int t = mine ? static_cast<int>(threadIdx.x) : per_token - 1;
  const int c = t % GROUP, h = t / GROUP;
  float sum[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) sum[k] = 0.f;
  const uint16_t* g = is_k ? g_k : g_q;
  const uint4 gain_a = *reinterpret_cast<const uint4*>(g + 8 * c), gain_b = *reinterpret_cast<const uint4*>(g + half + 8 * c);

  // one token: x, dy in shared memory (this thread's first half at 0, second at `half`)
  auto one = [&](const uint16_t* x, const uint16_t* dy, uint16_t* out, const float* cosv, const float* sinv) {
    float xa[8], xb[8], za[8], zb[8], ga[8], gb[8];
    load8<F>(x, 0, xa);
    load8<F>(x + half, 0, xb);
    load8<F>(dy, 0, za);
    load8<F>(dy + half, 0, zb);
    load8<FMT_BF16>(&gain_a, 0, ga);
    load8<FMT_BF16>(&gain_b, 0, gb);
    float ss = 0.f, dot = 0.f;
#pragma unroll
    for (int k4 = 0; k4 < 8; k4 += 4) {
      const float4 c4 = *reinterpret_cast<const float4*>(cosv + 8 * c + k4);
      const float4 s4 = *reinterpret_cast<const float4*>(sinv + 8 * c + k4);
      const float cs[4] = {c4.x, c4.y, c4.z, c4.w}, sn[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int k = k4 + q;
        const float a = za[k] * cs[q] + zb[k] * sn[q], b = zb[k] * cs[q] - za[k] * sn[q];  // R^T dy
        ss = fmaf(xa[k], xa[k], fmaf(xb[k], xb[k], ss));
        dot = fmaf(a * ga[k], xa[k], fmaf(b * gb[k], xb[k], dot));
        za[k] = a;
        zb[k] = b;
      }
    }
#pragma unroll
    for (int o = GROUP / 2; o > 0; o >>= 1) {
      ss += __shfl_xor_sync(0xffffffffu, ss, o);
      dot += __shfl_xor_sync(0xffffffffu, dot, o);
    }
    const float r = rsqrtf(ss * (1.f / HD) + eps);
    const float m = dot * (1.f / HD) * r * r;  // xh mean(du xh) = x m
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      sum[k] = fmaf(za[k], xa[k] * r, sum[k]);
      sum[8 + k] = fmaf(zb[k], xb[k] * r, sum[8 + k]);
      za[k] = r * fmaf(-m, xa[k], za[k] * ga[k]);
      zb[k] = r * fmaf(-m, xb[k], zb[k] * gb[k]);
    }
    if (mine) {
      store8<F, false>(out, 0, za);
      store8<F, false>(out + half, 0, zb);
    }
  };

  int u = 0;
  TokenWalk w(seq);
  for (int64_t bs = blockIdx.x; bs < tokens; bs += gridDim.x, w.step(seq)) {
    uint16_t* out = dx + bs * ld_dx + col + h * HD + 8 * c;
    if (w.s >= rope_count(ra, w.b)) {  // the whole CTA agrees
      if (mine) {
        const uint4 z = make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint4*>(out) = z;
        *reinterpret_cast<uint4*>(out + half) = z;
      }
      continue;
    }
    const int st = u % stages;
    // a wait that gave up has set the error word and every later one gives up soon; the warp's lanes go on
    // together, since they meet in every token's reduction, but do not free a slot whose copies may be on their way
    const bool got = mbar_wait(&full[st], static_cast<uint32_t>(u / stages) & 1u, guard, &abort_flag,
                               where_code(ERR_TIMEOUT_QKBWD, 2, u));
    const uint16_t* x = reinterpret_cast<const uint16_t*>(ring + st * 2 * row_bytes) + h * HD + 8 * c;
    one(x, x + d, out, s_cos[st], s_sin[st]);
    __syncwarp();
    if (lane == 0 && got) mbar_arrive(&empty[st]);
    ++u;
  }
  __syncthreads();  // every warp is done with the ring, and its copies have landed

  // sum over the CTA's heads: lanes of one warp that share c, then the warps
  float* s_red = reinterpret_cast<float*>(ring);
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    float v = mine ? sum[k] : 0.f;
#pragma unroll
    for (int o = 16; o >= GROUP; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane < GROUP) s_red[warp * HD + (k < 8 ? 0 : half) + 8 * lane + (k & 7)] = v;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < HD; i += 32 * warps) {
    float v = 0.f;
    for (int k = 0; k < warps; ++k) v += s_red[k * HD + i];
    part[blockIdx.x * static_cast<int64_t>(2 * HD) + (is_k ? HD : 0) + i] = v;
  }
}

// ------------------------------------------------------------------ RMSNorm rows

// r = (mean x^2 + eps)^(-1/2): dg_i = sum over rows of dy_i x_i r, and
// dx_i = r (dy_i g_i - x_i r^2 mean(dy g x)) + dres_i.  Both sums of a row come from one reduction; the
// gain and its gradient's sums stay in registers.
template <int F>
constexpr int bytes_of() {
  return F == FMT_F32 ? 4 : 2;
}

// Rows of up to 1024 columns: a warp per row, V vectors of 8 per lane; the next row is loaded before the
// current one's arithmetic and kept as it is in memory.  HBM-bound: event-timed with the sums' kernel, L2
// cold, 65536 rows: 1024 columns bf16 81 us (403 MB, 5.0 TB/s; the form for longer rows, whose CTA meets
// once per row, 130), 512 bf16 48 us (4.2 TB/s), 256 bf16 31 us (3.2 TB/s) and fp32 with dres 52 us
// (5.1 TB/s).  CTAs per SM: as many as hold the registers; at V = 1 three beat two in 16 bits (31 us
// against 34) and lose to them in fp32 (54 against 52).
constexpr int row_ctas(int v, bool fp32) { return v == 4 ? 1 : v == 2 || fp32 ? 2 : 3; }

template <int V, int XF, int DF, int OF>
__global__ void __launch_bounds__(256, row_ctas(V, XF == FMT_F32 || DF == FMT_F32))
    rmsnorm_bwd_warp_kernel(const void* __restrict__ x, const uint16_t* __restrict__ g, const void* __restrict__ dy,
                            const void* dres, void* dx, float* __restrict__ part, int64_t rows, int64_t cols,
                            float eps) {
  __shared__ __align__(16) float s_acc[8][V * 256];
  pdl_wait_then_release();
  const int nv = static_cast<int>(cols / 8), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float inv = 1.f / static_cast<float>(cols);
  const int64_t step = 8ll * gridDim.x;
  // 8 values as they are in memory
  constexpr int NX = bytes_of<XF>() / 2, NY = bytes_of<DF>() / 2;
  uint4 gr[V], xr[V][NX], yr[V][NY];
  float acc[V][8];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int64_t i = row * nv + lane + 32 * j;
      const bool in = lane + 32 * j < nv && row < rows;
#pragma unroll
      for (int k = 0; k < NX; ++k) xr[j][k] = in ? reinterpret_cast<const uint4*>(x)[i * NX + k] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int k = 0; k < NY; ++k) yr[j][k] = in ? reinterpret_cast<const uint4*>(dy)[i * NY + k] : make_uint4(0u, 0u, 0u, 0u);
    }
  };
#pragma unroll
  for (int j = 0; j < V; ++j) {
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[j][k] = 0.f;
    gr[j] = lane + 32 * j < nv ? reinterpret_cast<const uint4*>(g)[lane + 32 * j] : make_uint4(0u, 0u, 0u, 0u);
  }
  fetch(blockIdx.x * 8ll + warp);
#pragma unroll 1
  for (int64_t row = blockIdx.x * 8ll + warp; row < rows; row += step) {
    float xv[V][8], yv[V][8], e[V][8];
    float ss = 0.f, dot = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      load8<XF>(xr[j], 0, xv[j]);
      load8<DF>(yr[j], 0, yv[j]);
      float gv[8];
      load8<FMT_BF16>(&gr[j], 0, gv);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        ss = fmaf(xv[j][k], xv[j][k], ss);
        e[j][k] = 0.f;
        dot = fmaf(yv[j][k] * gv[k], xv[j][k], dot);
      }
      if (dres != nullptr && lane + 32 * j < nv) load8<OF>(dres, row * nv + lane + 32 * j, e[j]);
    }
    fetch(row + step);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      ss += __shfl_xor_sync(0xffffffffu, ss, o);
      dot += __shfl_xor_sync(0xffffffffu, dot, o);
    }
    const float r = rsqrtf(ss * inv + eps);
    const float m = dot * inv * r * r;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float gv[8];
      load8<FMT_BF16>(&gr[j], 0, gv);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        acc[j][k] = fmaf(yv[j][k], xv[j][k] * r, acc[j][k]);
        e[j][k] = fmaf(r, fmaf(-m, xv[j][k], yv[j][k] * gv[k]), e[j][k]);
      }
      if (lane + 32 * j < nv) store8<OF, false>(dx, row * nv + lane + 32 * j, e[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < V; ++j) store8<FMT_F32>(s_acc[warp], lane + 32 * j, acc[j]);
  __syncthreads();
  for (int i = threadIdx.x; i < cols; i += 256) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) v += s_acc[w][i];
    part[blockIdx.x * cols + i] = v;
  }
}

// Longer rows: a CTA per row at a time, V vectors of 8 per thread.  HBM-bound: x, dy and dres come
// through a ring of bulk copies that keeps up to 200 KB in flight per SM.  With the sums' kernel, event-timed,
// L2 cold: 4608 x 4096 fp32 rows with f16 dy 56 us (264 MB, 4.7 TB/s), bf16 41 us (151 MB, 3.6 TB/s), 16896 x 4096
// bf16 111 us (5.0 TB/s), 4608 x 8192 bf16 58 us (5.2 TB/s).  From registers with one row fetched ahead the same took
// 56, 44, 117 and 85 us.  A stage is free for its next row when the CTA has
// met in the following row's reduction.
template <int V, int XF, int DF, int OF>
__global__ void __launch_bounds__(512, V == 1 ? 2 : 1)
    rmsnorm_bwd_kernel(const void* __restrict__ x, const uint16_t* __restrict__ g, const void* __restrict__ dy,
                       const void* dres, void* dx, float* __restrict__ part, int64_t rows, int64_t cols, float eps,
                       int stages, const KernelGuard guard) {
  __shared__ __align__(16) float2 red[2][16];  // entries past the CTA's warps stay zero
  __shared__ uint64_t full[MAX_STAGES];
  __shared__ uint32_t abort_flag;
  extern __shared__ __align__(16) uint8_t ring[];  // [stages][x | dy | dres]
  const int nv = static_cast<int>(cols / 8);
  const uint32_t xb = static_cast<uint32_t>(cols) * bytes_of<XF>(), yb = static_cast<uint32_t>(cols) * bytes_of<DF>(),
                 eb = dres != nullptr ? static_cast<uint32_t>(cols) * bytes_of<OF>() : 0u;
  const uint32_t stage_bytes = xb + yb + eb;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float inv = 1.f / static_cast<float>(cols);
  if (threadIdx.x < 32) red[threadIdx.x >> 4][threadIdx.x & 15] = make_float2(0.f, 0.f);
  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) mbar_init(&full[i], 1);
    abort_flag = 0u;
    fence_barrier_init();
  }
  __syncthreads();
  pdl_wait_then_release();
  int issued = 0;  // thread 0
  auto load = [&](int64_t row) {
    const int st = issued % stages;
    uint8_t* at = ring + static_cast<size_t>(st) * stage_bytes;
    mbar_arrive_expect_tx(&full[st], stage_bytes);
    bulk_load(at, static_cast<const uint8_t*>(x) + row * xb, xb, &full[st]);
    bulk_load(at + xb, static_cast<const uint8_t*>(dy) + row * yb, yb, &full[st]);
    if (eb > 0) bulk_load(at + xb + yb, static_cast<const uint8_t*>(dres) + row * eb, eb, &full[st]);
    ++issued;
  };
  if (threadIdx.x == 0) {
    int64_t row = blockIdx.x;
    for (int i = 0; i < stages && row < rows; ++i, row += gridDim.x) load(row);
  }
  float gv[V][8], acc[V][8];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int i = threadIdx.x + j * blockDim.x;
#pragma unroll
    for (int k = 0; k < 8; ++k) gv[j][k] = acc[j][k] = 0.f;
    if (i < nv) load8<FMT_BF16>(g, i, gv[j]);
  }
  int u = 0;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x, ++u) {
    const int st = u % stages, buf = u & 1;
    // a thread whose wait gave up goes on to the row's barrier, whose verdict is the whole CTA's (a flag carried
    // along, or a vote of each warp, cost 9 % at 4608 x 4096 fp32 rows; the barrier's own vote 1 %)
    const bool got = mbar_wait(&full[st], static_cast<uint32_t>(u / stages) & 1u, guard, &abort_flag,
                    where_code(ERR_TIMEOUT_NORMBWD, 0, u));
    const uint8_t* at = ring + static_cast<size_t>(st) * stage_bytes;
    float xv[V][8], yv[V][8];
    float ss = 0.f, dot = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int i = threadIdx.x + j * blockDim.x;
#pragma unroll
      for (int k = 0; k < 8; ++k) xv[j][k] = yv[j][k] = 0.f;
      if (i < nv) {
        load8<XF>(at, i, xv[j]);
        load8<DF>(at + xb, i, yv[j]);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        ss = fmaf(xv[j][k], xv[j][k], ss);
        dot = fmaf(yv[j][k] * gv[j][k], xv[j][k], dot);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      ss += __shfl_xor_sync(0xffffffffu, ss, o);
      dot += __shfl_xor_sync(0xffffffffu, dot, o);
    }
    if (lane == 0) red[buf][warp] = make_float2(ss, dot);
    // two buffers: the next row's writes cannot meet this row's reads
    if (!__syncthreads_and(got)) break;
    // the CTA is done with the row before this one: its stage takes the row `stages` after it
    if (threadIdx.x == 0 && u > 0) {
      const int64_t ahead = row + (stages - 1) * static_cast<int64_t>(gridDim.x);
      if (ahead < rows) load(ahead);
    }
    ss = dot = 0.f;
#pragma unroll
    for (int w = 0; w < 16; w += 2) {
      const float4 v = *reinterpret_cast<const float4*>(&red[buf][w]);
      ss += v.x + v.z;
      dot += v.y + v.w;
    }
    const float r = rsqrtf(ss * inv + eps);
    const float m = dot * inv * r * r;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int i = threadIdx.x + j * blockDim.x;
      if (i >= nv) break;
      float o[8], e[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) e[k] = 0.f;
      if (eb > 0) load8<OF>(at + xb + yb, i, e);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        acc[j][k] = fmaf(yv[j][k], xv[j][k] * r, acc[j][k]);
        o[k] = fmaf(r, fmaf(-m, xv[j][k], yv[j][k] * gv[j][k]), e[k]);
      }
      store8<OF, false>(dx, row * nv + i, o);
    }
  }
  if (threadIdx.x == 0) {  // never leave with copies in flight
    for (int v = issued > stages ? issued - stages : 0; v < issued; ++v)
      mbar_wait(&full[v % stages], static_cast<uint32_t>(v / stages) & 1u, guard, &abort_flag,
                where_code(ERR_TIMEOUT_NORMBWD, 1, v), true);
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int i = threadIdx.x + j * blockDim.x;
    if (i < nv) store8<FMT_F32>(part, blockIdx.x * static_cast<int64_t>(nv) + i, acc[j]);
  }
}

// CTAs per SM of the long-row kernel, and the grid of all forms.
static int norm_ctas_per_sm(int64_t cols) { return cols <= 4096 ? 2 : 1; }
static int norm_grid(int64_t rows, int64_t cols, bool fp32) {
  const bool by_warps = cols <= 1024;
  const int64_t want = by_warps ? (rows + 7) / 8 : rows;
  const int64_t most =
      static_cast<int64_t>(SMS) * (by_warps ? row_ctas(cols <= 256 ? 1 : cols <= 512 ? 2 : 4, fp32) : norm_ctas_per_sm(cols));
  return static_cast<int>(want < most ? want : most);
}

template <int XF, int DF, int OF>
static cudaError_t launch_norm(const void* x, const uint16_t* g, const void* dy, const void* dres, void* dx,
                               float* part, int64_t rows, int64_t cols, float eps, int grid, const KernelGuard& guard,
                               cudaStream_t s) {
  const int nv = static_cast<int>(cols / 8);
  auto by_warps = [&](auto v) {
    return launch_pdl(rmsnorm_bwd_warp_kernel<decltype(v)::value, XF, DF, OF>, dim3(grid), dim3(256), 0, s, x, g, dy, dres,
                      dx, part, rows, cols, eps);
  };
  if (cols <= 256) return by_warps(std::integral_constant<int, 1>());
  if (cols <= 512) return by_warps(std::integral_constant<int, 2>());
  if (cols <= 1024) return by_warps(std::integral_constant<int, 4>());
  const int64_t stage = cols * (bytes_of<XF>() + bytes_of<DF>() + (dres != nullptr ? bytes_of<OF>() : 0));
  int64_t stages = 212 * 1024 / norm_ctas_per_sm(cols) / stage;
  stages = stages < 2 ? 2 : stages > MAX_STAGES ? MAX_STAGES : stages;
  const int smem = static_cast<int>(stages * stage);
  auto run = [&](auto v) {
    constexpr int V = decltype(v)::value;
    const cudaError_t e = allow_smem<rmsnorm_bwd_kernel<V, XF, DF, OF>>(smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(rmsnorm_bwd_kernel<V, XF, DF, OF>, dim3(grid), dim3(((nv + V - 1) / V + 31) / 32 * 32), smem, s, x,
                      g, dy, dres, dx, part, rows, cols, eps, static_cast<int>(stages), guard);
  };
  return nv <= 512 ? run(std::integral_constant<int, 1>()) : run(std::integral_constant<int, 2>());
}

template <int XF, int DF, typename... A>
static cudaError_t launch_norm_of(int dx_fmt, A... a) {
  if (dx_fmt == FMT_BF16) return launch_norm<XF, DF, FMT_BF16>(a...);
  if (dx_fmt == FMT_F16) return launch_norm<XF, DF, FMT_F16>(a...);
  return launch_norm<XF, DF, FMT_F32>(a...);
}

template <int XF, typename... A>
static cudaError_t launch_norm_df(int dy_fmt, int dx_fmt, A... a) {
  if (dy_fmt == FMT_BF16) return launch_norm_of<XF, FMT_BF16>(dx_fmt, a...);
  if (dy_fmt == FMT_F16) return launch_norm_of<XF, FMT_F16>(dx_fmt, a...);
  return launch_norm_of<XF, FMT_F32>(dx_fmt, a...);
}

// CTAs of the QK-norm gradient for each of q and k.
static int qk_grid(int64_t tokens, int per_token) {
  const int64_t most = qk_ctas(per_token) * SMS / 2;
  return static_cast<int>(tokens < most ? tokens : most);
}

}  // namespace tew

size_t qknorm_mrope_bwd_workspace(int64_t tokens, int n_heads, int head_dim) {
  return static_cast<size_t>(tew::qk_grid(tokens, n_heads * (head_dim / 16))) * 2 * head_dim * 4;
}

cudaError_t launch_qknorm_mrope_bwd(const void* qkv, Rows dqk, Rows dx, float* dg_q, float* dg_k, int fmt, int batch,
                                    int seq, int n_heads, int head_dim, int n_text, int grid_w, int n_img, int t_img,
                                    const int32_t* pos, const int32_t* text_lens, const int32_t sections[3],
                                    float theta, const uint16_t* g_q, const uint16_t* g_k, float eps, void* workspace,
                                    const KernelGuard& guard, cudaStream_t s) {
  const int64_t tokens = static_cast<int64_t>(batch) * seq;
  const int per_token = n_heads * (head_dim / 16);
  if (per_token > 512) return cudaErrorInvalidValue;  // the kernel's launch bound
  const RopeArgs ra = rope_args(n_text, grid_w, n_img, t_img, pos, text_lens, nullptr, sections, theta, head_dim);
  const int warps = (per_token + 31) / 32;
  const int grid = tew::qk_grid(tokens, per_token);
  // a stage holds the raw rows and their gradients; an SM's CTAs share about 190 KB
  const int stage = 4 * n_heads * head_dim;
  int stages = 190 * 1024 / tew::qk_ctas(per_token) / stage;
  stages = stages < 2 ? 2 : stages > tew::MAX_STAGES ? tew::MAX_STAGES : stages;
  const int sums = warps * head_dim * 4;
  const int smem = stages * stage > sums ? stages * stage : sums;
  float* part = static_cast<float*>(workspace);
  auto run = [&](auto fm, auto hd, auto most) {
    constexpr auto kern = tew::qknorm_mrope_bwd_kernel<decltype(fm)::value, decltype(hd)::value, decltype(most)::value>;
    const cudaError_t e = allow_smem<kern>(smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(grid, 2), dim3(32 * (warps + 2)), smem, s, static_cast<const uint16_t*>(qkv),
                      static_cast<const uint16_t*>(dqk.p), dqk.ld, static_cast<uint16_t*>(const_cast<void*>(dx.p)),
                      dx.ld, part, tokens, seq, n_heads, ra, g_q, g_k, eps, stages, guard);
  };
  auto of = [&](auto hd) {
    const std::integral_constant<int, 256> two_per_sm;
    const std::integral_constant<int, 512> one_per_sm;
    const std::integral_constant<int, FMT_F16> f16;
    const std::integral_constant<int, FMT_BF16> bf16;
    if (per_token <= 256) return fmt == FMT_F16 ? run(f16, hd, two_per_sm) : run(bf16, hd, two_per_sm);
    return fmt == FMT_F16 ? run(f16, hd, one_per_sm) : run(bf16, hd, one_per_sm);
  };
  cudaError_t e;
  if (head_dim == 128)
    e = of(std::integral_constant<int, 128>());
  else if (head_dim == 64)
    e = of(std::integral_constant<int, 64>());
  else
    return cudaErrorInvalidValue;
  if (e != cudaSuccess) return e;
  return tew::sum_rows(part, grid, 2 * head_dim, dg_q, dg_k, head_dim, s);
}

size_t rmsnorm_bwd_workspace(int64_t rows, int64_t cols) {
  return static_cast<size_t>(tew::norm_grid(rows, cols, false)) * static_cast<size_t>(cols) * 4;  // no fewer CTAs than with fp32
}

cudaError_t launch_rmsnorm_bwd(const void* x, int x_fmt, const uint16_t* g, const void* dy, int dy_fmt,
                               const void* dres, void* dx, int dx_fmt, float* dg, int64_t rows, int64_t cols,
                               float eps, void* workspace, const KernelGuard& guard, cudaStream_t s) {
  const int grid = tew::norm_grid(rows, cols, x_fmt == FMT_F32 || dy_fmt == FMT_F32);
  float* part = static_cast<float*>(workspace);
  cudaError_t e;
  if (x_fmt == FMT_BF16)
    e = tew::launch_norm_df<FMT_BF16>(dy_fmt, dx_fmt, x, g, dy, dres, dx, part, rows, cols, eps, grid, guard, s);
  else
    e = tew::launch_norm_df<FMT_F32>(dy_fmt, dx_fmt, x, g, dy, dres, dx, part, rows, cols, eps, grid, guard, s);
  if (e != cudaSuccess) return e;
  return tew::sum_rows(part, grid, cols, dg, dg, cols, s);
}

}  // namespace jab
