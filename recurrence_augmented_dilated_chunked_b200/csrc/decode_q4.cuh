// decode_q4.cuh -- the D-compressed cache with its dilated rows held in 4
// bits: prefill hand-off, read-back, and the fused decode step over it.
//
// A row of Dh channels is kept in groups of 32 channels.  A group holds its
// minimum m (a bf16 input's minimum is exact in bf16), the step s =
// bf16((max - min) / 15) and one code per channel, n = rint((x - m) / s)
// clamped to 0..15 (0 where s == 0), so the row stands for m + n s.  That is
// Dh/2 + Dh/8 bytes for a row against 2 Dh in bf16 (80 against 256 for Dh =
// 128).  Codes: one 32-bit word per 8 channels; channel c of the word sits in
// nibble c/2 + 4 (c mod 2), so that (w >> 4i) & 0x000f000f is the pair of
// neighbouring channels 2i, 2i + 1 as two 16-bit halves.  Parameters: one
// word per group, s in the low half, m in the high half.  The window ring
// stays bf16 and the recurrent state fp32.
//
// Decode step: the grid, the split of a (b, h)'s virtual key list over CTAs,
// the recurrence in split 0 and the closing merge are those of decode.cuh.
// The step is bound by the cache's bytes, but a row that shrank 3.2x leaves
// only ~28 issue slots per key at the memory rate, and expanding 2 x 128
// codes in fp32 arithmetic costs about as many.  So the products run as
// m16n8k16 bf16 MMAs, whose operands are one shift-and-mask per code pair:
// 0x4300 | n is the bf16 number 128 + n exactly.
//   scores  A = 16 keys x 16 channels of codes.  Lane (g, t) of a warp (g =
//           lane / 4, t = lane % 4) holds keys g and g + 8, channels
//           [t Dh/4, (t + 1) Dh/4).  B's column n is q restricted to quarter
//           n of the channels, so C[key][n] are the quarters' separate dot
//           products, and the score is sum_n s_n C[key][n] + (m_n - 128 s_n)
//           sum(q in quarter n) (a quarter is one group for Dh = 128, half a
//           group for Dh = 64).  q enters as it is (bf16), sums are fp32.
//   values  A = 16 channels x 16 keys of codes (two keys' halves merged by a
//           byte permute).  B's columns 0..3 are the keys' weights p s of each
//           quarter, split into a bf16 part (columns 0..3) and the bf16 rest
//           (columns 4..7), so a weight keeps 16 bits; the offset 128 and the
//           minima are taken out in fp32 against those same parts.
// Ring rows are bf16 already and go through the same accumulators with
// weights p.
#pragma once
#include "common.cuh"
#include "decode.cuh"

namespace ratp {
namespace decode_q4 {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 16;          // keys per warp step
constexpr int kGroup = 32;         // channels per scale
// A ring key moves 512 bytes where a 4-bit key moves 160: it counts as three
// when a (b, h)'s keys are split over CTAs.
constexpr int kRingUnits = 3;
constexpr int kPrefetchRows = 128; // rows per split warmed into L2 before the wait

struct Params {
  decode::Params d;                // Kc / Vc hold codes (see codes())
  uint32_t* Kp;                    // [B][rows_per_b][Dh / 32]
  uint32_t* Vp;
};

template <int DH>
struct Row {
  static constexpr int kWords = DH / 8;        // code words
  static constexpr int kParams = DH / kGroup;  // parameter words
};

__device__ __forceinline__ float param_scale(uint32_t p) { return __uint_as_float(p << 16); }
__device__ __forceinline__ float param_min(uint32_t p) { return __uint_as_float(p & 0xffff0000u); }

// ---- quantisation -------------------------------------------------------------
// IEEE division and rounding to nearest even throughout, so the codes are the
// definition's.
__device__ __forceinline__ uint32_t group_params(float lo, float hi) {
  const __nv_bfloat16 s = __float2bfloat16_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.f));
  const __nv_bfloat16 m = __float2bfloat16_rn(lo);   // exact: lo is a bf16 value
  return (uint32_t)__bfloat16_as_ushort(s) | ((uint32_t)__bfloat16_as_ushort(m) << 16);
}
__device__ __forceinline__ uint32_t code_of(float x, uint32_t par) {
  const float s = param_scale(par);
  if (!(s > 0.f)) return 0u;
  const float n = rintf(__fdiv_rn(__fsub_rn(x, param_min(par)), s));
  return (uint32_t)fminf(fmaxf(n, 0.f), 15.f);
}
__device__ __forceinline__ int nibble_shift(int c) { return 4 * ((c >> 1) + 4 * (c & 1)); }

// 8 consecutive channels of a row -> one code word; the 4 lanes of a group of
// 32 channels (consecutive, aligned) share its parameters.  All 4 call.
__device__ __forceinline__ uint32_t quantise8(const float* f, uint32_t* par, unsigned lanes) {
  float lo = f[0], hi = f[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) { lo = fminf(lo, f[i]); hi = fmaxf(hi, f[i]); }
#pragma unroll
  for (int off = 1; off < 4; off <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(lanes, lo, off));
    hi = fmaxf(hi, __shfl_xor_sync(lanes, hi, off));
  }
  *par = group_params(lo, hi);
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) w |= code_of(f[i], *par) << nibble_shift(i);
  return w;
}

// ---- prefill -> cache hand-off ------------------------------------------------
struct PackParams {
  decode::PackParams d;
  uint32_t* Kp;
  uint32_t* Vp;
};

// The grid and row numbering of decode::pack_kernel: Dh/8 threads per row,
// dilated rows first (quantised), then the ring rows (copied).
template <int DH>
__global__ void __launch_bounds__(256)
pack_kernel(const PackParams pp) {
  const decode::PackParams& p = pp.d;
  constexpr int TPR = DH / 8;
  constexpr int RPB = 256 / TPR;
  const int h = blockIdx.y, b = blockIdx.z;
  const int r = blockIdx.x * RPB + threadIdx.x / TPR;
  const int li = threadIdx.x % TPR;
  const bool dense = decode::is_dense(p.dense_bits, h);
  const int Dd = dense ? 1 : p.D;
  const int n_dil = p.T / Dd;
  const int w_lo = max(0, p.T - p.W);
  const int n_ring = (p.W > 0) ? (p.T - w_lo) : 0;
  if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0) p.len[b] = p.T;
  const long long src_base = (long long)b * p.T * p.H * DH + (long long)h * DH + li * 8;
  [[maybe_unused]] const long long n_src = (long long)p.B * p.T * p.H * DH;
  const unsigned lanes = 0xfu << ((threadIdx.x & 31) & ~3);
  if (r < n_dil) {
    const long long src = src_base + ((long long)r * Dd + Dd - 1) * p.H * DH;
    const long long row = (long long)b * p.rows_per_b + decode::head_offset(p.dense_bits, h, p.T_max, p.D) + r;
    if (!RATP_IN(src, 8, n_src) || !RATP_IN(row, 1, (long long)p.B * p.rows_per_b)) return;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      float f[8];
      uint32_t par;
      Elem<__nv_bfloat16>::unpack(__ldcs(reinterpret_cast<const uint4*>((s == 0 ? p.hk : p.hv) + src)), f);
      const uint32_t w = quantise8(f, &par, lanes);
      reinterpret_cast<uint32_t*>(s == 0 ? p.Kc : p.Vc)[row * (DH / 8) + li] = w;
      if ((li & 3) == 0) (s == 0 ? pp.Kp : pp.Vp)[row * (DH / kGroup) + li / 4] = par;
    }
  } else if (r < n_dil + n_ring) {
    const int pos = w_lo + (r - n_dil);
    const long long src = src_base + (long long)pos * p.H * DH;
    const long long dst = (((long long)b * p.H + h) * p.W + pos % p.W) * DH + li * 8;
    if (!RATP_IN(src, 8, n_src) || !RATP_IN(dst, 8, (long long)p.B * p.H * p.W * DH)) return;
    *reinterpret_cast<uint4*>(p.Kw + dst) = *reinterpret_cast<const uint4*>(p.hk + src);
    *reinterpret_cast<uint4*>(p.Vw + dst) = *reinterpret_cast<const uint4*>(p.hv + src);
  }
}

// ---- read-back: the values that the held rows stand for, fp32 ------------------
// One thread per code word (8 channels): out[row][8 w .. 8 w + 7].
__global__ void __launch_bounds__(256)
unpack_kernel(const uint32_t* __restrict__ codes, const uint32_t* __restrict__ params, float* __restrict__ out,
              long long words) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= words) return;
  const uint32_t w = __ldcs(codes + i), par = params[i >> 2];
  const float s = param_scale(par), m = param_min(par);
  float f[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) f[c] = __fadd_rn(m, __fmul_rn((float)((w >> nibble_shift(c)) & 15u), s));
  float4* o = reinterpret_cast<float4*>(out) + 2 * i;
  __stcs(o, make_float4(f[0], f[1], f[2], f[3]));
  __stcs(o + 1, make_float4(f[4], f[5], f[6], f[7]));
}

// ---- decode -------------------------------------------------------------------
__device__ __forceinline__ void mma_bf16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Code pairs of a word as bf16 pairs 128 + n (channels 2i, 2i + 1).
__device__ __forceinline__ uint32_t pair_of(uint32_t w, int i) { return ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u; }

// One tile of up to 16 keys as a warp holds it: lane (g, t) has the K words of
// keys g, g + 8 (its channel quarter) and the V words of keys t, 4 + t, 8 + t,
// 12 + t (channels [g Dh/8, (g + 1) Dh/8)), with the parameters it needs.
template <int DH>
struct Tile4 {
  static constexpr int NW = DH / 64 * 2;       // K words per key and lane (16 or 32 channels)
  static constexpr int NV = DH / 64;           // V words per key and lane (8 or 16 channels)
  uint32_t k[2][NW];
  uint32_t kp[2][2];                           // lanes t < 2: quarters 2t, 2t + 1
  uint32_t v[4][NV];
  uint32_t vp[4];                              // quarter g % 4
};

template <int N>
__device__ __forceinline__ void load_words(uint32_t* r, const uint32_t* src) {
  if constexpr (N == 4) {
    const uint4 x = __ldcs(reinterpret_cast<const uint4*>(src));
    r[0] = x.x; r[1] = x.y; r[2] = x.z; r[3] = x.w;
  } else if constexpr (N == 2) {
    const uint2 x = __ldcs(reinterpret_cast<const uint2*>(src));
    r[0] = x.x; r[1] = x.y;
  } else {
    r[0] = __ldcs(src);
  }
}

template <int DH>
__device__ __forceinline__ void load_tile(Tile4<DH>& f, const uint32_t* kc, const uint32_t* kp, const uint32_t* vc,
                                          const uint32_t* vp, int n, int g, int t) {
  constexpr int W = DH / 8, P = DH / kGroup;
  constexpr int NW = Tile4<DH>::NW, NV = Tile4<DH>::NV;
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int key = g + 8 * r;
#pragma unroll
    for (int i = 0; i < NW; ++i) f.k[r][i] = 0;
    f.kp[r][0] = f.kp[r][1] = 0;
    if (key < n) {
      load_words<NW>(f.k[r], kc + key * W + t * NW);
      if (t < 2) {
        if constexpr (P == 4) load_words<2>(f.kp[r], kp + key * P + 2 * t);
        else f.kp[r][0] = f.kp[r][1] = __ldcs(kp + key * P + t);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int key = 4 * j + t;
#pragma unroll
    for (int i = 0; i < NV; ++i) f.v[j][i] = 0;
    f.vp[j] = 0;
    if (key < n) {
      load_words<NV>(f.v[j], vc + key * W + g * NV);
      f.vp[j] = __ldcs(vp + key * P + (g & 3) * P / 4);
    }
  }
}

// Running softmax of one warp: m, l (this lane's share) and the accumulators.
template <int DH>
struct Acc {
  float m, l;
  float z;                 // this lane's column: fp32 share of the minima and offsets
  float c[DH / 16][4];     // MMA j: channels 2 of this lane's Dh/8 x columns
};

// Scores of the tile's keys g, g + 8 (log2 units; -inf past n) into the
// softmax: rescales on a new maximum, returns the weights.
template <int DH>
__device__ __forceinline__ void weigh(Acc<DH>& a, float s0, float s1, int n, int g, float* p0, float* p1) {
  s0 = g < n ? s0 : -INFINITY;
  s1 = g + 8 < n ? s1 : -INFINITY;
  float m = fmaxf(s0, s1);
#pragma unroll
  for (int off = 4; off < 32; off <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  m = fmaxf(m, a.m);
  if (m > a.m) {           // the whole warp agrees
    const float r = exp2f(a.m - m);
    a.l *= r;
    a.z *= r;
#pragma unroll
    for (int j = 0; j < DH / 16; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) a.c[j][i] *= r;
    a.m = m;
  }
  *p0 = m == -INFINITY ? 0.f : exp2f(s0 - m);
  *p1 = m == -INFINITY ? 0.f : exp2f(s1 - m);
  a.l += *p0 + *p1;
}

// Weights of this lane's column for keys t, 4 + t, 8 + t, 12 + t: column < 4
// the bf16 part, column >= 4 the bf16 rest of w.
__device__ __forceinline__ float part_of(float w, int g) {
  const float hi = __bfloat162float(__float2bfloat16_rn(w));
  return g < 4 ? hi : __bfloat162float(__float2bfloat16_rn(w - hi));
}

template <int DH>
__device__ __forceinline__ void attend_codes(Acc<DH>& a, const Tile4<DH>& f, const uint32_t (*qf)[2], const float* qsum,
                                             float scale_log2, int n, int g, int t) {
  constexpr int NW = Tile4<DH>::NW, NV = Tile4<DH>::NV;
  float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < 2 * NW; ++j) {           // 4 channels of each quarter per MMA
    const int w = j / 2, i = 2 * (j % 2);
    mma_bf16(d, pair_of(f.k[0][w], i), pair_of(f.k[1][w], i), pair_of(f.k[0][w], i + 1), pair_of(f.k[1][w], i + 1),
             qf[j][0], qf[j][1]);
  }
  // lanes t = 0, 1 hold quarters (0, 1) and (2, 3); the others' columns are unused
  float s[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const float sa = param_scale(f.kp[r][0]), sb = param_scale(f.kp[r][1]);
    float x = fmaf(sa, d[2 * r], fmaf(sb, d[2 * r + 1], 0.f));
    x = fmaf(fmaf(-128.f, sa, param_min(f.kp[r][0])), qsum[0], x);
    x = fmaf(fmaf(-128.f, sb, param_min(f.kp[r][1])), qsum[1], x);
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    s[r] = __shfl_sync(0xffffffffu, x, 0, 4) * scale_log2;
  }
  float p0, p1;
  weigh(a, s[0], s[1], n, g, &p0, &p1);
  // this lane's column weights for keys t, 4 + t, 8 + t, 12 + t
  float pw[4] = {__shfl_sync(0xffffffffu, p0, 4 * t), __shfl_sync(0xffffffffu, p0, 16 + 4 * t),
                 __shfl_sync(0xffffffffu, p1, 4 * t), __shfl_sync(0xffffffffu, p1, 16 + 4 * t)};
  float x[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[j] = part_of(pw[j] * param_scale(f.vp[j]), g);
    a.z = fmaf(-128.f, x[j], a.z);
    if (g < 4) a.z = fmaf(pw[j], param_min(f.vp[j]), a.z);
  }
  const uint32_t b0 = pack_bf16x2(x[0], x[1]), b1 = pack_bf16x2(x[2], x[3]);
#pragma unroll
  for (int w = 0; w < NV; ++w) {
    // low halves: channels 0, 2, 4, 6 of the word; high halves: 1, 3, 5, 7
    const uint32_t l01 = __byte_perm(f.v[0][w], f.v[1][w], 0x5410), h01 = __byte_perm(f.v[0][w], f.v[1][w], 0x7632);
    const uint32_t l23 = __byte_perm(f.v[2][w], f.v[3][w], 0x5410), h23 = __byte_perm(f.v[2][w], f.v[3][w], 0x7632);
#pragma unroll
    for (int i = 0; i < 4; ++i)                // channels 2i (row g) and 2i + 1 (row g + 8)
      mma_bf16(a.c[4 * w + i], pair_of(l01, i), pair_of(h01, i), pair_of(l23, i), pair_of(h23, i), b0, b1);
  }
}

// The same with bf16 ring rows; rows are passed by address, at most n of 16
// (key j of the tile is ring position pos0 + j).
template <int DH>
__device__ __forceinline__ void attend_ring(Acc<DH>& a, const __nv_bfloat16* kw, const __nv_bfloat16* vw, int pos0, int W,
                                            const uint32_t (*qf)[2], float scale_log2, int n, int g, int t) {
  constexpr int NW = Tile4<DH>::NW, NV = Tile4<DH>::NV;
  float d[4] = {0.f, 0.f, 0.f, 0.f};
  uint4 kr[2][NW];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int key = g + 8 * r;
#pragma unroll
    for (int i = 0; i < NW; ++i)
      kr[r][i] = key < n ? __ldcs(reinterpret_cast<const uint4*>(kw + (long long)((pos0 + key) % W) * DH + t * (DH / 4)) + i)
                         : make_uint4(0u, 0u, 0u, 0u);
  }
  uint4 vr[4][NV];
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int i = 0; i < NV; ++i)
      vr[j][i] = 4 * j + t < n
                     ? __ldcs(reinterpret_cast<const uint4*>(vw + (long long)((pos0 + 4 * j + t) % W) * DH + g * (DH / 8)) + i)
                     : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    mma_bf16(d, kr[0][w].x, kr[1][w].x, kr[0][w].y, kr[1][w].y, qf[2 * w][0], qf[2 * w][1]);
    mma_bf16(d, kr[0][w].z, kr[1][w].z, kr[0][w].w, kr[1][w].w, qf[2 * w + 1][0], qf[2 * w + 1][1]);
  }
  float s[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    float x = d[2 * r] + d[2 * r + 1];
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    s[r] = __shfl_sync(0xffffffffu, x, 0, 4) * scale_log2;
  }
  float p0, p1;
  weigh(a, s[0], s[1], n, g, &p0, &p1);
  float pw[4] = {__shfl_sync(0xffffffffu, p0, 4 * t), __shfl_sync(0xffffffffu, p0, 16 + 4 * t),
                 __shfl_sync(0xffffffffu, p1, 4 * t), __shfl_sync(0xffffffffu, p1, 16 + 4 * t)};
#pragma unroll
  for (int j = 0; j < 4; ++j) pw[j] = part_of(pw[j], g);
  const uint32_t b0 = pack_bf16x2(pw[0], pw[1]), b1 = pack_bf16x2(pw[2], pw[3]);
#pragma unroll
  for (int w = 0; w < NV; ++w) {
    const uint32_t y[4][4] = {{vr[0][w].x, vr[0][w].y, vr[0][w].z, vr[0][w].w},
                              {vr[1][w].x, vr[1][w].y, vr[1][w].z, vr[1][w].w},
                              {vr[2][w].x, vr[2][w].y, vr[2][w].z, vr[2][w].w},
                              {vr[3][w].x, vr[3][w].y, vr[3][w].z, vr[3][w].w}};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      mma_bf16(a.c[4 * w + i], __byte_perm(y[0][i], y[1][i], 0x5410), __byte_perm(y[0][i], y[1][i], 0x7632),
               __byte_perm(y[2][i], y[3][i], 0x5410), __byte_perm(y[2][i], y[3][i], 0x7632), b0, b1);
  }
}

template <int DH>
__global__ void __launch_bounds__(kThreads)
decode_kernel(const Params pp) {
  const decode::Params& p = pp.d;
  constexpr int W8 = DH / 8, PG = DH / kGroup;
  constexpr int NQ = DH / 16;                  // score MMAs per tile
  constexpr int NE = kWarps + 1;               // merged entries: the warps and the query's own key
  constexpr int kStride = kWarps * kTile;

  __shared__ __align__(16) float s_self[2][DH];
  __shared__ float s_m[NE], s_l[NE];
  __shared__ __align__(16) float s_acc[NE][DH];
  __shared__ int s_last;

  const int b = blockIdx.x / p.splits_per_b;
  const int rem = blockIdx.x - b * p.splits_per_b;
  const int h = decode::head_of_split(p, rem);
  const int split = rem - p.split_base[h];
  const int tid = threadIdx.x;
  const bool dense = decode::is_dense(p.dense_bits, h);
  const int cap = dense ? p.T_max : p.T_max / p.D;
  const long long row0 = (long long)b * p.rows_per_b + decode::head_offset(p.dense_bits, h, p.T_max, p.D);
  [[maybe_unused]] const long long n_rows = (long long)p.B * p.rows_per_b;
  uint32_t* const kc = reinterpret_cast<uint32_t*>(p.Kc);
  uint32_t* const vc = reinterpret_cast<uint32_t*>(p.Vc);

  // as in decode.cuh: let the next step be scheduled, warm L2 with this
  // split's first rows, then wait for the kernels before this one
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == 0) {
    const int first = min(split * p.split_keys, cap);
    const int n = min(kPrefetchRows, cap - first);
    if (n > 0 && RATP_IN(row0 + first, n, n_rows)) {
      decode::bulk_prefetch_l2(kc + (row0 + first) * W8, (uint32_t)n * W8 * 4);
      decode::bulk_prefetch_l2(vc + (row0 + first) * W8, (uint32_t)n * W8 * 4);
      if (PG % 4 == 0) {                       // a parameter row of 16 bytes
        decode::bulk_prefetch_l2(pp.Kp + (row0 + first) * PG, (uint32_t)n * PG * 4);
        decode::bulk_prefetch_l2(pp.Vp + (row0 + first) * PG, (uint32_t)n * PG * 4);
      }
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int t = p.len[b];
  const int Dd = dense ? 1 : p.D;
  bool active = true;
  int n_slots = 0, w_lo = 0, n_win = 0, n_used = 1, app_slot = 0;
  if (t >= p.T_max) {
    active = false;
    if (split == 0 && h == 0 && tid == 0) raise_error(RATP_ERR_CAPACITY);
  } else {
    app_slot = t / Dd;
    n_slots = app_slot;
    if (p.W > 0 && !dense) {
      w_lo = max(0, t - p.W + 1);
      n_win = t - w_lo;
      n_slots = w_lo / Dd;                     // dilated slots before the window
    }
    const long long units = n_slots + (long long)kRingUnits * n_win;
    n_used = (int)max(1ll, (units + p.split_keys - 1) / p.split_keys);
    if (split >= n_used) active = false;
  }

  if (active) {
    const long long bh = (long long)b * p.H + h;
    [[maybe_unused]] const long long n_tok = (long long)p.B * p.H * DH;
    [[maybe_unused]] const long long n_ring = (long long)p.B * p.H * p.W * DH;
    const int warp = tid >> 5, lane = tid & 31, g = lane >> 2, tq = lane & 3;

    if (split == 0) {
      decode::recurrence_step<DH>(p, bh, t, s_self[0], s_self[1], [](int, int, __nv_bfloat16) {});
      if (t % Dd == Dd - 1) {
        if (app_slot >= cap) {
          if (tid == 0) raise_error(RATP_ERR_CAPACITY);
        } else if (tid < 2 * W8 && RATP_IN(row0 + app_slot, 1, n_rows)) {
          // 8 channels per thread; W8 threads per stream, in whole groups of 4
          const int st = tid / W8, w = tid % W8;
          uint32_t par;
          const uint32_t code = quantise8(&s_self[st][8 * w], &par, 0xfu << (lane & ~3));
          (st == 0 ? kc : vc)[(row0 + app_slot) * W8 + w] = code;
          if ((w & 3) == 0) (st == 0 ? pp.Kp : pp.Vp)[(row0 + app_slot) * PG + w / 4] = par;
        }
      }
    }

    // ---- the query: fragments of this lane's channel quarter, quarter sums ----
    uint32_t qf[NQ][2];
    float qsum[2];
    const bool q_ok = RATP_IN(bh * DH, DH, n_tok);
    {
      const uint4* q4 = reinterpret_cast<const uint4*>(p.q + bh * DH + tq * (DH / 4));
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < DH / 32; ++i) {
        const uint4 v = q_ok ? q4[i] : make_uint4(0u, 0u, 0u, 0u);
        float f[8];
        Elem<__nv_bfloat16>::unpack(v, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum += f[j];
        const bool mine = g == tq;             // B's column n = g is quarter n alone
        qf[2 * i][0] = mine ? v.x : 0u;
        qf[2 * i][1] = mine ? v.y : 0u;
        qf[2 * i + 1][0] = mine ? v.z : 0u;
        qf[2 * i + 1][1] = mine ? v.w : 0u;
      }
      qsum[0] = __shfl_sync(0xffffffffu, sum, 2 * tq, 4);          // quarters 2t, 2t + 1 (used by t < 2)
      qsum[1] = __shfl_sync(0xffffffffu, sum, 2 * tq + 1, 4);
    }

    Acc<DH> a;
    a.m = -INFINITY;
    a.l = 0.f;
    a.z = 0.f;
#pragma unroll
    for (int j = 0; j < NQ; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) a.c[j][i] = 0.f;

    // ---- this split's share: units [u0, u1) of slots, then of ring keys ----
    const long long u0 = (long long)split * p.split_keys, u1 = u0 + p.split_keys;
    const int s_end = (int)min((long long)n_slots, u1);
    const auto ring_at = [&](long long u) {
      return (int)min((long long)n_win, (max(u - n_slots, 0ll) + kRingUnits - 1) / kRingUnits);
    };
    int k = (int)min((long long)n_slots, u0) + warp * kTile;
    Tile4<DH> cur;
    auto load = [&](Tile4<DH>& f, int at) {
      int n = min(kTile, s_end - at);
      if (!RATP_IN(row0 + at, max(n, 0), n_rows)) n = 0;
      load_tile<DH>(f, kc + (row0 + at) * W8, pp.Kp + (row0 + at) * PG, vc + (row0 + at) * W8,
                    pp.Vp + (row0 + at) * PG, n, g, tq);
    };
    if (k < s_end) load(cur, k);
    while (k < s_end) {
      Tile4<DH> next;
      const int kn = k + kStride;
      if (kn < s_end) load(next, kn);
      attend_codes<DH>(a, cur, qf, qsum, p.scale_log2, min(kTile, s_end - k), g, tq);
      cur = next;
      k = kn;
    }
    const int r_end = ring_at(u1);
    if (n_win > 0 && RATP_IN(bh * p.W * DH, (long long)p.W * DH, n_ring)) {
      const __nv_bfloat16* kw = p.Kw + bh * p.W * DH;
      const __nv_bfloat16* vw = p.Vw + bh * p.W * DH;
      for (int r = ring_at(u0) + warp * kTile; r < r_end; r += kStride)
        attend_ring<DH>(a, kw, vw, w_lo + r, p.W, qf, p.scale_log2, min(kTile, r_end - r), g, tq);
    }

    // ---- this warp's entry ----
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) a.l += __shfl_xor_sync(0xffffffffu, a.l, off);
    a.z += __shfl_xor_sync(0xffffffffu, a.z, 1);
    a.z += __shfl_xor_sync(0xffffffffu, a.z, 2);
    a.z += __shfl_xor_sync(0xffffffffu, a.z, 16);                  // lanes g and g + 4: quarter g % 4
    const float z = __shfl_sync(0xffffffffu, a.z, (g >> 1) << 2);  // of the quarter this lane's channels lie in
    if (lane == 0) { s_m[warp] = a.m; s_l[warp] = a.l; }
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
      // columns g / 2 (lane t = g / 4) and 4 + g / 2 (lane t = 2 + g / 4)
      const bool odd = (g >> 1) & 1;
      float x0 = odd ? a.c[j][1] : a.c[j][0], x1 = odd ? a.c[j][3] : a.c[j][2];
      x0 += __shfl_xor_sync(0xffffffffu, x0, 2);
      x1 += __shfl_xor_sync(0xffffffffu, x1, 2);
      if (tq == (g >> 2)) {
        const int ch = g * (DH / 8) + 2 * j;   // MMA j = 4 w + i: channels 8 w + 2 i, + 1
        *reinterpret_cast<float2*>(&s_acc[warp][ch]) = make_float2(x0 + z, x1 + z);
      }
    }
    // ---- the query's own key, an entry of its own in split 0 ----
    if (warp == 0) {
      float s = -INFINITY;
      if (split == 0) {
        s = 0.f;
        if (q_ok)
          for (int c = lane; c < DH; c += 32) s = fmaf(__bfloat162float(p.q[bh * DH + c]), s_self[0][c], s);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        s *= p.scale_log2;
      }
      if (lane == 0) { s_m[kWarps] = s; s_l[kWarps] = split == 0 ? 1.f : 0.f; }
      for (int c = lane; c < DH; c += 32) s_acc[kWarps][c] = split == 0 ? s_self[1][c] : 0.f;
    }
    __syncthreads();
    decode::merge_entries<DH, NE>(p, bh, split, n_used, s_m, s_l, s_acc, &s_last);
  }

  decode::advance_len(p, b);
}

}  // namespace decode_q4
}  // namespace ratp
