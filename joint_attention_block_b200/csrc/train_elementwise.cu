// HBM-bound gradients: QK-RMSNorm + 3D M-RoPE and the row RMSNorm, each with the sums of its
// gains' gradients.  fp32 math.  The sums are taken in a fixed order (registers over a CTA's
// tokens or rows, then shared memory, then one partial row per CTA that a second kernel adds up), so
// a result does not change from run to run.
#include "common.cuh"
#include "rope.cuh"
#include "train.h"

namespace jab {
namespace tew {

constexpr int MAX_CTAS = 296;  // two per SM: what the workspaces hold a partial row for

// dst[c] = sum over the n rows of part [n, cols]; one CTA per 32 columns, 32 row lanes each.
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

// ------------------------------------------------------------------ QK-RMSNorm + M-RoPE

// With x a raw head vector, r = (mean x^2 + eps)^(-1/2), xh = r x, u = xh g and y = R u (R the
// token's rotation of the pairs (i, i + hd/2)): dz = R^T dy, dg = sum dz xh, du = dz g and
// dx = r (du - xh mean(du xh)).
// Thread layout as in the forward kernel (one thread per head and 8 rotary pairs, q and k); each
// CTA walks tokens with the gains' sums in registers, the next token's vectors loaded and its
// angles computed (the other of two shared buffers) before the current token's arithmetic.
// Tokens behind an element's count are not read; their gradients are zeros.
template <int F, int HD>
__global__ void __launch_bounds__(512)
    qknorm_mrope_bwd_kernel(const uint16_t* __restrict__ qkv, const uint16_t* dqk, int64_t ld_dqk, uint16_t* dx,
                            int64_t ld_dx, float* __restrict__ part, int64_t tokens, int seq, int n_heads, RopeArgs ra,
                            const uint16_t* __restrict__ g_q, const uint16_t* __restrict__ g_k, float eps) {
  constexpr int half = HD / 2;
  constexpr int GROUP = HD / 16;  // threads per head
  __shared__ float s_cos[2][half], s_sin[2][half];
  __shared__ int s_live[2];
  extern __shared__ float s_red[];  // [warps][2 HD]
  pdl_wait_then_release();
  const int per_token = n_heads * GROUP;
  const bool mine = static_cast<int>(threadIdx.x) < per_token;
  const int t = mine ? static_cast<int>(threadIdx.x) : per_token - 1;
  const int c = t % GROUP, h = t / GROUP;
  const int d = n_heads * HD;

  struct Vecs {
    uint4 v[8];  // raw q (two halves), raw k, gradient of q, gradient of k
  };
  auto load = [&](int64_t bs, Vecs& w) {
    const uint16_t* x = qkv + bs * 3 * d + h * HD + 8 * c;
    const uint16_t* g = dqk + bs * ld_dqk + h * HD + 8 * c;
    w.v[0] = *reinterpret_cast<const uint4*>(x);
    w.v[1] = *reinterpret_cast<const uint4*>(x + half);
    w.v[2] = *reinterpret_cast<const uint4*>(x + d);
    w.v[3] = *reinterpret_cast<const uint4*>(x + d + half);
    w.v[4] = *reinterpret_cast<const uint4*>(g);
    w.v[5] = *reinterpret_cast<const uint4*>(g + half);
    w.v[6] = *reinterpret_cast<const uint4*>(g + d);
    w.v[7] = *reinterpret_cast<const uint4*>(g + d + half);
  };
  auto angles = [&](int64_t bs, int buf) {
    const int b = static_cast<int>(bs / seq), s = static_cast<int>(bs - static_cast<int64_t>(b) * seq);
    int pt, ph, pw;
    const int count = rope_position(ra, b, s, pt, ph, pw);
    if (threadIdx.x == 0) s_live[buf] = s < count;
    for (int i = threadIdx.x; i < half; i += blockDim.x)
      rope_angle(ra, i, i < ra.sec_t ? pt : (i < ra.sec_t + ra.sec_h ? ph : pw), s_cos[buf][i], s_sin[buf][i]);
  };
  float acc[2][16];
#pragma unroll
  for (int k = 0; k < 16; ++k) acc[0][k] = acc[1][k] = 0.f;

  int64_t bs = blockIdx.x;
  Vecs cur;
  if (bs < tokens) {
    load(bs, cur);
    angles(bs, 0);
  }
  __syncthreads();
  for (int buf = 0; bs < tokens; bs += gridDim.x, buf ^= 1) {
    const int64_t next = bs + gridDim.x;
    Vecs nxt;
    if (next < tokens) {
      load(next, nxt);
      angles(next, buf ^ 1);
    } else {
      nxt = cur;
    }
    uint16_t* out = dx + bs * ld_dx + h * HD + 8 * c;
    const bool live = s_live[buf] != 0;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const uint16_t* g = w == 0 ? g_q : g_k;
      float ga[8], gb[8], xa[8], xb[8], da[8], db[8];
      load8<FMT_BF16>(g + 8 * c, 0, ga);
      load8<FMT_BF16>(g + half + 8 * c, 0, gb);
      load8<F>(&cur.v[2 * w], 0, xa);
      load8<F>(&cur.v[2 * w + 1], 0, xb);
      load8<F>(&cur.v[4 + 2 * w], 0, da);
      load8<F>(&cur.v[4 + 2 * w + 1], 0, db);
      float ss = 0.f, dot = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float cs = s_cos[buf][8 * c + k], sn = s_sin[buf][8 * c + k];
        const float za = da[k] * cs + db[k] * sn, zb = db[k] * cs - da[k] * sn;  // R^T dy
        ss = fmaf(xa[k], xa[k], fmaf(xb[k], xb[k], ss));
        dot = fmaf(za * ga[k], xa[k], fmaf(zb * gb[k], xb[k], dot));
        da[k] = za;
        db[k] = zb;
      }
#pragma unroll
      for (int o = GROUP / 2; o > 0; o >>= 1) {
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
        dot += __shfl_xor_sync(0xffffffffu, dot, o);
      }
      const float r = rsqrtf(ss * (1.f / HD) + eps);
      const float m = dot * (1.f / HD) * r * r;  // xh mean(du xh) = x m
      float oa[8], ob[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (live) {
          acc[w][k] = fmaf(da[k], xa[k] * r, acc[w][k]);
          acc[w][8 + k] = fmaf(db[k], xb[k] * r, acc[w][8 + k]);
        }
        oa[k] = live ? r * fmaf(-m, xa[k], da[k] * ga[k]) : 0.f;
        ob[k] = live ? r * fmaf(-m, xb[k], db[k] * gb[k]) : 0.f;
      }
      if (mine) {
        store8<F>(out + w * d, 0, oa);
        store8<F>(out + w * d + half, 0, ob);
      }
    }
    cur = nxt;
    __syncthreads();  // the next token's angles are written, this token's are read
  }

  // sum over the CTA's heads: lanes of one warp that share c, then the warps
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      float v = mine ? acc[w][k] : 0.f;
#pragma unroll
      for (int o = 16; o >= GROUP; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane < GROUP) s_red[warp * 2 * HD + w * HD + (k < 8 ? 0 : half) + 8 * lane + (k & 7)] = v;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * HD; i += blockDim.x) {
    float v = 0.f;
    for (int k = 0; k < warps; ++k) v += s_red[k * 2 * HD + i];
    part[blockIdx.x * static_cast<int64_t>(2 * HD) + i] = v;
  }
}

// ------------------------------------------------------------------ RMSNorm rows

// r = (mean x^2 + eps)^(-1/2): dg_i = sum over rows of dy_i x_i r, and
// dx_i = r (dy_i g_i - x_i r^2 mean(dy g x)) + dres_i.
// One row per CTA at a time, both of its sums in one reduction; V vectors of 8 per thread, whose
// gain, gain sums and row stay in registers; the next row is loaded before the reduction.
template <int F>
struct Raw8 {
  uint4 v[F == FMT_F32 ? 2 : 1];
};
template <int F>
__device__ __forceinline__ Raw8<F> fetch8(const void* p, int64_t i8) {
  Raw8<F> r;
  constexpr int N = F == FMT_F32 ? 2 : 1;
#pragma unroll
  for (int k = 0; k < N; ++k) r.v[k] = reinterpret_cast<const uint4*>(p)[N * i8 + k];
  return r;
}

template <int V, int XF, int DF, int OF>
__global__ void __launch_bounds__(512)
    rmsnorm_bwd_kernel(const void* __restrict__ x, const uint16_t* __restrict__ g, const void* __restrict__ dy,
                       const void* dres, void* dx, float* __restrict__ part, int64_t rows, int64_t cols, float eps) {
  __shared__ float2 red[2][16];
  pdl_wait_then_release();
  const int nv = static_cast<int>(cols / 8);
  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float inv = 1.f / static_cast<float>(cols);
  float gv[V][8], acc[V][8];
  Raw8<XF> rx[V];
  Raw8<DF> ry[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int i = threadIdx.x + j * blockDim.x;
#pragma unroll
    for (int k = 0; k < 8; ++k) gv[j][k] = acc[j][k] = 0.f;
    rx[j] = Raw8<XF>{};
    ry[j] = Raw8<DF>{};
    if (i < nv) {
      load8<FMT_BF16>(g, i, gv[j]);
      if (blockIdx.x < rows) {
        rx[j] = fetch8<XF>(x, blockIdx.x * static_cast<int64_t>(nv) + i);
        ry[j] = fetch8<DF>(dy, blockIdx.x * static_cast<int64_t>(nv) + i);
      }
    }
  }
  int buf = 0;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x, buf ^= 1) {
    const int64_t next = row + gridDim.x;
    float xv[V][8], yv[V][8];
    float ss = 0.f, dot = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      load8<XF>(rx[j].v, 0, xv[j]);
      load8<DF>(ry[j].v, 0, yv[j]);
      const int i = threadIdx.x + j * blockDim.x;
      if (i < nv && next < rows) {
        rx[j] = fetch8<XF>(x, next * nv + i);
        ry[j] = fetch8<DF>(dy, next * nv + i);
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
    __syncthreads();  // two buffers: the next row's writes cannot meet this row's reads
    ss = dot = 0.f;
    for (int w = 0; w < warps; ++w) {
      ss += red[buf][w].x;
      dot += red[buf][w].y;
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
      if (dres != nullptr) load8<OF>(dres, row * nv + i, e);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        acc[j][k] = fmaf(yv[j][k], xv[j][k] * r, acc[j][k]);
        o[k] = fmaf(r, fmaf(-m, xv[j][k], yv[j][k] * gv[j][k]), e[k]);
      }
      store8<OF>(dx, row * nv + i, o);
    }
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int i = threadIdx.x + j * blockDim.x;
    if (i < nv) store8<FMT_F32>(part, blockIdx.x * static_cast<int64_t>(nv) + i, acc[j]);
  }
}

template <int XF, int DF, int OF>
static cudaError_t launch_norm(const void* x, const uint16_t* g, const void* dy, const void* dres, void* dx,
                               float* part, int64_t rows, int64_t cols, float eps, int grid, cudaStream_t s) {
  const int nv = static_cast<int>(cols / 8);
  if (nv <= 512)
    return launch_pdl(rmsnorm_bwd_kernel<1, XF, DF, OF>, dim3(grid), dim3((nv + 31) / 32 * 32), 0, s, x, g, dy, dres,
                      dx, part, rows, cols, eps);
  return launch_pdl(rmsnorm_bwd_kernel<2, XF, DF, OF>, dim3(grid), dim3(((nv + 1) / 2 + 31) / 32 * 32), 0, s, x, g, dy,
                    dres, dx, part, rows, cols, eps);
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

static int ctas(int64_t n) { return static_cast<int>(n < MAX_CTAS ? n : MAX_CTAS); }

}  // namespace tew

size_t qknorm_mrope_bwd_workspace(int64_t tokens, int head_dim) {
  return static_cast<size_t>(tew::ctas(tokens)) * 2 * head_dim * 4;
}

cudaError_t launch_qknorm_mrope_bwd(const void* qkv, Rows dqk, Rows dx, float* dg_q, float* dg_k, int fmt, int batch,
                                    int seq, int n_heads, int head_dim, int n_text, int grid_w, int n_img, int t_img,
                                    const int32_t* pos, const int32_t* text_lens, const int32_t sections[3],
                                    float theta, const uint16_t* g_q, const uint16_t* g_k, float eps, void* workspace,
                                    cudaStream_t s) {
  const int64_t tokens = static_cast<int64_t>(batch) * seq;
  const int per_token = n_heads * (head_dim / 16);
  if (per_token > 512) return cudaErrorInvalidValue;  // the kernel's launch bound
  const RopeArgs ra = rope_args(n_text, grid_w, n_img, t_img, pos, text_lens, nullptr, sections, theta, head_dim);
  const int threads = (per_token + 31) / 32 * 32;
  const int grid = tew::ctas(tokens);
  float* part = static_cast<float*>(workspace);
  auto run = [&](auto kern) {
    return launch_pdl(kern, dim3(grid), dim3(threads), static_cast<size_t>(threads / 32) * 2 * head_dim * 4, s,
                      static_cast<const uint16_t*>(qkv), static_cast<const uint16_t*>(dqk.p), dqk.ld,
                      static_cast<uint16_t*>(const_cast<void*>(dx.p)), dx.ld, part, tokens, seq, n_heads, ra, g_q, g_k,
                      eps);
  };
  cudaError_t e;
  if (head_dim == 128)
    e = fmt == FMT_F16 ? run(tew::qknorm_mrope_bwd_kernel<FMT_F16, 128>)
                       : run(tew::qknorm_mrope_bwd_kernel<FMT_BF16, 128>);
  else if (head_dim == 64)
    e = fmt == FMT_F16 ? run(tew::qknorm_mrope_bwd_kernel<FMT_F16, 64>)
                       : run(tew::qknorm_mrope_bwd_kernel<FMT_BF16, 64>);
  else
    return cudaErrorInvalidValue;
  if (e != cudaSuccess) return e;
  return tew::sum_rows(part, grid, 2 * head_dim, dg_q, dg_k, head_dim, s);
}

size_t rmsnorm_bwd_workspace(int64_t rows, int64_t cols) {
  return static_cast<size_t>(tew::ctas(rows)) * static_cast<size_t>(cols) * 4;
}

cudaError_t launch_rmsnorm_bwd(const void* x, int x_fmt, const uint16_t* g, const void* dy, int dy_fmt,
                               const void* dres, void* dx, int dx_fmt, float* dg, int64_t rows, int64_t cols,
                               float eps, void* workspace, cudaStream_t s) {
  const int grid = tew::ctas(rows);
  float* part = static_cast<float*>(workspace);
  cudaError_t e;
  if (x_fmt == FMT_BF16)
    e = tew::launch_norm_df<FMT_BF16>(dy_fmt, dx_fmt, x, g, dy, dres, dx, part, rows, cols, eps, grid, s);
  else
    e = tew::launch_norm_df<FMT_F32>(dy_fmt, dx_fmt, x, g, dy, dres, dx, part, rows, cols, eps, grid, s);
  if (e != cudaSuccess) return e;
  return tew::sum_rows(part, grid, cols, dg, dg, cols, s);
}

}  // namespace jab
