// Positions and angles of the 3D rotary embedding, shared by the QK-norm kernel and its gradient.
#pragma once

#include <cmath>

#include "common.cuh"

namespace jab {

// Text token j -> (j, j, j); image cell (r, c) in raster order -> (t_img, r, c).
// Positions and inverse frequencies of the rotary embedding, passed by value to the kernels.
struct RopeArgs {
  int n_text, grid_w, n_img, t_img;  // t_img < 0: n_text (or L_b in a padded batch)
  const int32_t* pos;                // [S, 3] or NULL (ignored when text_lens is given)
  const int32_t* text_lens;          // [batch] or NULL
  int32_t* kv_len;                   // [batch] or NULL: receives L_b + n_img
  int sec_t, sec_h;                  // rotary pairs on the t and h axes (w takes the rest)
  float inv_freq[64];                // fp32(theta^(-2i/hd)), i < hd/2
};

inline RopeArgs rope_args(int n_text, int grid_w, int n_img, int t_img, const int32_t* pos, const int32_t* text_lens,
                          int32_t* kv_len, const int32_t sections[3], float theta, int head_dim) {
  RopeArgs ra;
  ra.n_text = n_text;
  ra.grid_w = grid_w > 0 ? grid_w : 1;
  ra.n_img = n_img;
  ra.t_img = t_img;
  ra.pos = pos;
  ra.text_lens = text_lens;
  ra.kv_len = kv_len;
  ra.sec_t = sections[0];
  ra.sec_h = sections[1];
  for (int i = 0; i < head_dim / 2; ++i)
    ra.inv_freq[i] = static_cast<float>(std::pow(static_cast<double>(theta), -2.0 * i / head_dim));
  return ra;
}

__device__ __forceinline__ void token_position(int s, int n_text, int grid_w, int t_img, const int32_t* pos, int& pt,
                                               int& ph, int& pw) {
  if (pos != nullptr) {
    pt = pos[3 * s];
    ph = pos[3 * s + 1];
    pw = pos[3 * s + 2];
  } else if (s < n_text) {
    pt = ph = pw = s;
  } else {
    const int i = s - n_text;
    pt = t_img;
    ph = i / grid_w;
    pw = i - ph * grid_w;
  }
}

// Tokens of element b that take part.
__device__ __forceinline__ int rope_count(const RopeArgs& ra, int b) {
  return (ra.text_lens != nullptr ? min(max(ra.text_lens[b], 0), ra.n_text) : ra.n_text) + ra.n_img;
}

// Position of token s of element b; returns the number of tokens of the element that take part
// (padding rows beyond it sit at (0, 0, 0)).
__device__ __forceinline__ int rope_position(const RopeArgs& ra, int b, int s, int& pt, int& ph, int& pw) {
  if (ra.text_lens != nullptr) {
    const int L = min(max(ra.text_lens[b], 0), ra.n_text);
    pt = ph = pw = 0;
    if (s < L) {
      pt = ph = pw = s;
    } else if (s < L + ra.n_img) {
      const int k = s - L;
      pt = ra.t_img < 0 ? L : ra.t_img;
      ph = k / ra.grid_w;
      pw = k - ph * ra.grid_w;
    }
    return L + ra.n_img;
  }
  token_position(s, ra.n_text, ra.grid_w, ra.t_img < 0 ? ra.n_text : ra.t_img, ra.pos, pt, ph, pw);
  return ra.n_text + ra.n_img;
}

// Cosine and sine of pair i's angle at position p on its axis: p * inv_freq_i is exact in fp64; it is
// reduced by the nearest multiple of 2 pi in fp64 (error ~1e-13 for the angles of any image),
// rounded once to fp32 in [-pi, pi], and its sine and cosine taken in fp32.
__device__ __forceinline__ void rope_angle(float inv_freq, int p, float& cs, float& sn) {
  const double x = static_cast<double>(p) * static_cast<double>(inv_freq);
  const double k = rint(x * 0.15915494309189535);
  const float r = static_cast<float>(fma(-k, 6.283185307179586, x));
  sincosf(r, &sn, &cs);
}

}  // namespace jab
