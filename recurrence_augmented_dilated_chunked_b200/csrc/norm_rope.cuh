// norm_rope.cuh -- RMS norm of every head of q and k with the rotary position
// in the same pass (the step between a layer's projections and its mixer: the
// scan and the attention at prefill, the decode step for a single token).
//
//   r = rsqrt(mean_c(x_c^2) + eps),  y_c = x_c r w_c          (per head, fp32)
//   pair i of the first `rot` channels: angle a = pos * inv_freq[i],
//   (u, v) -> (u cos a - v sin a, v cos a + u sin a)
// pair i is channels (i, i + rot/2), or (2i, 2i + 1) when interleaved; the
// channels from `rot` on are only normalised.
//
// Bound by memory: every element is read once and written once.  A group of
// Dh/8 lanes owns one token of one tensor and walks its heads, so the sines
// are computed once per token in registers: each lane holds two quads of four
// channels, chosen so that both members of a pair lie in the same lane (no
// shuffle but the norm's sum).  Two heads' rows are in flight per group and eight
// CTAs of 128 threads on an SM, 64 registers a thread: 4 x 8192 tokens of 32 + 32
// heads of 128 channels (1.07 GB) take 183 us in single calls and 196 us in a row,
// 5.9 and 5.5 TB/s (four heads in flight, or other occupancies: 190 to 245 us).
// The 64 registers spill 12 bytes a thread in bf16 and 52 in fp32 (20 and 72 loaded).
// Few tokens are bound by latency: 64 tokens of 16 + 16 heads take 4 us.
// The angle is formed and reduced to a fraction of a turn in 64 bits, since
// pos * inv_freq in 32 bits is off by whole radians at far positions.
#pragma once
#include "common.cuh"

namespace ratp {
namespace norm_rope {

constexpr int kThreads = 128;
constexpr int kUnroll = 2;      // heads in flight per group

struct Tensor {
  const void* x;
  void* y;
  const float* w;               // [Dh] gains, or NULL for 1
  long long xs_b, xs_t, xs_h;   // element strides; channels contiguous
  long long ys_b, ys_t, ys_h;
  int H;
  int n_blk;                    // head blocks per token
  int blk;                      // heads per block
};

struct Params {
  Tensor tensor[2];             // q, k
  const float* inv_freq;        // [rot / 2]
  const int32_t* pos;           // NULL, [B] (position of token 0) or [B][T]
  int pos_per_token;
  int B, T, rot, interleaved;
  float eps;
  long long units0, units;      // units of tensor 0, of both
};

template <typename E> struct Quad;
template <> struct Quad<__nv_bfloat16> {
  using V = uint2;
  __device__ static __forceinline__ void unpack(const V& v, float* f) {
    f[0] = __uint_as_float(v.x << 16); f[1] = __uint_as_float(v.x & 0xffff0000u);
    f[2] = __uint_as_float(v.y << 16); f[3] = __uint_as_float(v.y & 0xffff0000u);
  }
  __device__ static __forceinline__ V pack(const float* f) {
    return make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
  }
};
template <> struct Quad<float> {
  using V = float4;
  __device__ static __forceinline__ void unpack(const V& v, float* f) {
    f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
  }
  __device__ static __forceinline__ V pack(const float* f) { return make_float4(f[0], f[1], f[2], f[3]); }
};

template <typename E, int DH>
__global__ void __launch_bounds__(kThreads, 8)
norm_rope_kernel(const Params p) {
  using Q = Quad<E>;
  using V = typename Q::V;
  constexpr int G = DH / 8;                      // lanes per group
  const int li = threadIdx.x % G;
  const long long unit = (long long)blockIdx.x * (kThreads / G) + threadIdx.x / G;
  if (unit >= p.units) return;                   // whole groups leave; shuffles below name the group's lanes
  const unsigned lanes = (G == 32) ? 0xffffffffu : (((1u << (G & 31)) - 1u) << ((threadIdx.x & 31) / G * G));
  const int which = unit >= p.units0 ? 1 : 0;
  const Tensor& a = p.tensor[which];
  const long long u = which ? unit - p.units0 : unit;
  const long long tok = u / a.n_blk;
  const int h0 = (int)(u - tok * a.n_blk) * a.blk;
  const int h1 = min(a.H, h0 + a.blk);
  const long long b = tok / p.T;
  const long long t = tok - b * p.T;

  // this lane's two quads of channels, and pairs 4 li .. 4 li + 3
  const int rl = p.rot / 8;                      // lanes that rotate
  int qa, qb;
  if (li < rl) {
    qa = p.interleaved ? 2 * li : li;
    qb = p.interleaved ? 2 * li + 1 : li + rl;
  } else {
    qa = 2 * li;
    qb = 2 * li + 1;
  }
  const E* x = static_cast<const E*>(a.x) + b * a.xs_b + t * a.xs_t;
  E* y = static_cast<E*>(a.y) + b * a.ys_b + t * a.ys_t;
  // elements of the views, for the guarded build (strides are not negative)
  [[maybe_unused]] const long long xn = (p.B - 1) * a.xs_b + (p.T - 1) * a.xs_t + (a.H - 1) * a.xs_h + DH;
  [[maybe_unused]] const long long yn = (p.B - 1) * a.ys_b + (p.T - 1) * a.ys_t + (a.H - 1) * a.ys_h + DH;
  [[maybe_unused]] const long long xo = b * a.xs_b + t * a.xs_t, yo = b * a.ys_b + t * a.ys_t;

  V va[kUnroll], vb[kUnroll];
  auto load = [&](int h) {
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      if (h + i < h1 && RATP_IN(xo + (h + i) * a.xs_h, DH, xn)) {
        const E* r = x + (h + i) * a.xs_h;
        va[i] = *reinterpret_cast<const V*>(r + 4 * qa);
        vb[i] = *reinterpret_cast<const V*>(r + 4 * qb);
      } else {
        va[i] = V{};
        vb[i] = V{};
      }
    }
  };
  load(h0);

  float wa[4] = {1.f, 1.f, 1.f, 1.f}, wb[4] = {1.f, 1.f, 1.f, 1.f};
  if (a.w != nullptr) {
    Quad<float>::unpack(*reinterpret_cast<const float4*>(a.w + 4 * qa), wa);
    Quad<float>::unpack(*reinterpret_cast<const float4*>(a.w + 4 * qb), wb);
  }
  float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
  if (li < rl) {
    double pos = (double)t;
    if (p.pos != nullptr && RATP_IN(p.pos_per_token ? b * p.T + t : b, 1, p.pos_per_token ? (long long)p.B * p.T : p.B))
      pos = p.pos_per_token ? (double)p.pos[b * p.T + t] : pos + (double)p.pos[b];
    float fr[4];
    Quad<float>::unpack(*reinterpret_cast<const float4*>(p.inv_freq + 4 * li), fr);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const double turns = pos * (double)fr[i] * 0.15915494309189533577;   // 1 / (2 pi)
      sincospif((float)(2.0 * (turns - rint(turns))), &s[i], &c[i]);
    }
  }

  for (int h = h0; h < h1; h += kUnroll) {
    float f[kUnroll][8], ss[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      Q::unpack(va[i], f[i]);
      Q::unpack(vb[i], f[i] + 4);
      float2 acc = make_float2(0.f, 0.f);
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const float2 e = make_float2(f[i][j], f[i][j + 1]);
        acc = fma2(e, e, acc);
      }
      ss[i] = acc.x + acc.y;
    }
    const int hn = h + kUnroll;
    if (hn < h1) load(hn);                       // the next heads' rows, while these are finished
#pragma unroll
    for (int off = G / 2; off > 0; off >>= 1)
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) ss[i] += __shfl_xor_sync(lanes, ss[i], off);
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      if (h + i >= h1) continue;
      // fp32 outputs keep the root's last bits; bf16 has no place for them
      const float ms = ss[i] * (1.f / DH) + p.eps;
      const float r = sizeof(E) == 4 ? __frsqrt_rn(ms) : rsqrtf(ms);
      float oa[4], ob[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        oa[j] = f[i][j] * r * wa[j];
        ob[j] = f[i][4 + j] * r * wb[j];
      }
      if (!p.interleaved) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float ua = oa[j], ub = ob[j];
          oa[j] = fmaf(ua, c[j], -ub * s[j]);
          ob[j] = fmaf(ub, c[j], ua * s[j]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float ua = oa[2 * j], ub = oa[2 * j + 1], uc = ob[2 * j], ud = ob[2 * j + 1];
          oa[2 * j] = fmaf(ua, c[j], -ub * s[j]);
          oa[2 * j + 1] = fmaf(ub, c[j], ua * s[j]);
          ob[2 * j] = fmaf(uc, c[2 + j], -ud * s[2 + j]);
          ob[2 * j + 1] = fmaf(ud, c[2 + j], uc * s[2 + j]);
        }
      }
      if (RATP_IN(yo + (h + i) * a.ys_h, DH, yn)) {
        E* o = y + (h + i) * a.ys_h;
        *reinterpret_cast<V*>(o + 4 * qa) = Q::pack(oa);
        *reinterpret_cast<V*>(o + 4 * qb) = Q::pack(ob);
      }
    }
  }
}

}  // namespace norm_rope
}  // namespace ratp
