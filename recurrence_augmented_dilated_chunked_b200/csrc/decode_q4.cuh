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
// word per group, s in the low half, m in the high half.  The rows of 32
// consecutive slots of a head form a block (struct Block): its K codes, V codes,
// K parameters and V parameters one after the other, 5 KB for Dh = 128.  A block
// is what a warp fetches at a time, so the step reads memory in long pieces (four
// separate arrays streamed at 4.4 - 4.8 TB/s).  The window ring stays bf16 and the
// recurrent state fp32.
//
// Decode step: the grid, the split of a (b, h)'s virtual key list over CTAs,
// the recurrence in split 0 and the closing merge are those of decode.cuh.
// The step is bound by the cache's bytes, but a row that shrank 3.2x leaves
// only ~28 issue slots per key at the memory rate, and expanding 2 x 128
// codes in fp32 arithmetic costs about as many.  So the products run as
// m16n8k16 bf16 MMAs, whose operands are one shift-and-mask per code pair:
// 0x4180 | n << 3 is the bf16 number 16 + n exactly.
//   scores  A = 16 keys x 16 channels of codes.  Lane (g, t) of a warp (g =
//           lane / 4, t = lane % 4) holds keys g and g + 8, channels
//           [t Dh/4, (t + 1) Dh/4).  B's column n is q restricted to quarter
//           n of the channels, so C[key][n] are the quarters' separate dot
//           products, and the score is sum_n s_n C[key][n] + (m_n - 16 s_n)
//           sum(q in quarter n) (a quarter is one group for Dh = 128, half a
//           group for Dh = 64).  q enters as it is (bf16), sums are fp32.
//   values  A = 16 channels x 16 keys of codes (two keys' halves merged by a
//           byte permute).  B's columns 0..3 are the keys' weights p s of each
//           quarter, split into a bf16 part (columns 0..3) and the bf16 rest
//           (columns 4..7), so a weight keeps 16 bits.  A group's values are
//           m + 7.5 s (its middle, summed in fp32) and s (n - 7.5): the products
//           sum 16 + n, from which 23.5 times those same parts is taken every
//           kFold steps.  The sums' roundings go by their size, which is 23.5 p s
//           a key until then (tensor cores cut them off, always towards zero),
//           while the output of many keys alike is the small rest of values that
//           cancel: 256 keys between, at most 2^-23 of the sum lost by each
//           product, leave 2^-15 of a step s however long the split (128 + n,
//           taken out at the end only, was off by 1.0% of the output's norm in
//           splits of 3648 alike keys and by 44% in one of 32768; the rounding of
//           o is 0.16%).
// Ring rows are bf16 already and go through the same accumulators with
// weights p.
// Measured (floors at 6.55 TB/s): 64 sequences x 16 heads of 512 slots and a
// window of 128, 39.5 us of 23.5; 4 x 32 heads of 8192 slots, 47 us of 25.7.  About
// 10 us are the step's start and end (length, inputs, merge, closing counters);
// the rest is held by the expansion of the codes as much as by memory (the second
// case took 43 us without its fetches, 37 us without its products).  Ring rows by
// 16-byte copies of the lanes: 42 us for the first.
#pragma once
#include "common.cuh"
#include "decode.cuh"
#include "sm100.cuh"

#include <stddef.h>

namespace ratp {
namespace decode_q4 {

// Two warps per CTA: eight CTAs per SM hold more (b, h) at once than four of
// twice the size, and each has its own start and end to wait through.
constexpr int kThreads = 64;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 16;          // keys per MMA tile
constexpr int kStep = 32;          // cached rows per warp step
constexpr int kRingStep = 8;       // ring rows per warp step (their bytes fit the same stage)
constexpr int kStages = 2;         // steps in flight per warp (20 KB of blocks a CTA)
constexpr int kCtasPerSm = 8;      // 16 warps of 128 registers (with 7 and three stages 49 and 58 us)
constexpr int kGroup = 32;         // channels per scale
// A ring key moves 512 bytes where a 4-bit key moves 160: it counts as three
// when a (b, h)'s keys are split over CTAs.
constexpr int kRingUnits = 3;
constexpr int kPrefetchBlocks = 1; // blocks per split warmed into L2 before the wait

// kStep consecutive slots of one head: codes and parameters of K and V.
template <int DH>
struct Block {
  uint32_t k[kStep][DH / 8];
  uint32_t v[kStep][DH / 8];
  uint32_t kp[kStep][DH / kGroup];
  uint32_t vp[kStep][DH / kGroup];
};

__host__ __device__ constexpr long long blocks_of(long long cap) { return (cap + kStep - 1) / kStep; }

// First block of head h inside one batch item.
__device__ __forceinline__ long long head_block(const unsigned long long* bits, int h, int T_max, int D) {
  int nd = 0;
  for (int w = 0; w < (h >> 6); ++w) nd += __popcll(bits[w]);
  if (h & 63) nd += __popcll(bits[h >> 6] & ((1ull << (h & 63)) - 1ull));
  return nd * blocks_of(T_max) + (h - nd) * blocks_of(T_max / D);
}

struct Params {
  decode::Params d;                // Kc: Block<DH> [B][blocks_per_b]
  long long blocks_per_b;
};

__device__ __forceinline__ float param_scale(uint32_t p) { return __uint_as_float(p << 16); }
__device__ __forceinline__ float param_min(uint32_t p) { return __uint_as_float(p & 0xffff0000u); }

// ---- quantisation -------------------------------------------------------------
// Every step rounds as the definition does (to nearest even; x - m to fp32, the
// quotient of that by s once, to the code), so the codes are the definition's.
__device__ __forceinline__ uint32_t group_params(float lo, float hi) {
  // d / 15 correctly rounded: the product's remainder is exact in one fma, and
  // no quotient by 15 lies near enough to a rounding boundary to be missed
  const float d = __fsub_rn(hi, lo), q = __fmul_rn(d, 1.f / 15.f);
  if (!(d < INFINITY)) return 0x7fff7fffu;           // a value that is not finite: the group stands for NaN
  const __nv_bfloat16 s = __float2bfloat16_rn(__fmaf_rn(__fmaf_rn(-15.f, q, d), 1.f / 15.f, q));
  const __nv_bfloat16 m = __float2bfloat16_rn(lo);   // exact: lo is a bf16 value
  return (uint32_t)__bfloat16_as_ushort(s) | ((uint32_t)__bfloat16_as_ushort(m) << 16);
}
// rint(d / s) for d = x - m >= 0, as the integer added to 1.5 * 2^23 (its bits
// hold it): the product with an approximate reciprocal is at most one off, and
// the remainder d - n s, exact in one fma (n s has 12 bits), says where.  The
// quotient's own rounding to fp32 never makes a tie: two fp32 numbers d whose
// quotients by s straddle a tie lie further apart than half its last place.
constexpr float kIntBias = 12582912.f;
__device__ __forceinline__ uint32_t code_bits(float d, float s, float r) {
  float nb = __fadd_rn(__fmul_rn(d, r), kIntBias);
  const float n = nb - kIntBias;
  const float rem = __fmaf_rn(-n, s, d);
  const float twice = 2.f * fabsf(rem);
  const bool off = twice > s || (twice == s && (__float_as_uint(nb) & 1u));
  if (off) nb += copysignf(1.f, rem);
  return __float_as_uint(nb);
}
__device__ __forceinline__ int nibble_shift(int c) { return 4 * ((c >> 1) + 4 * (c & 1)); }

// 8 M consecutive channels of a row (bf16 pairs) -> M code words; the 4 / M lanes
// of a group of 32 channels (consecutive, aligned) share its parameters.  All of
// them call.  A code is first taken from the quotient's product d r snapped to a
// multiple of 2^-19 (2^-18 past 8) by the first addition, which makes exact
// ties exact again, and rounded to even by the second; the remainder shows the
// rare case of a quotient that near a tie that was none (x some 2^18 times
// smaller than the group's minimum), and the words are done over.
template <int M>
__device__ __forceinline__ void quantise(const uint4* x, uint32_t* words, uint32_t* par, unsigned lanes) {
  const uint32_t* v = reinterpret_cast<const uint32_t*>(x);
  __nv_bfloat162 lo2 = *reinterpret_cast<const __nv_bfloat162*>(&v[0]), hi2 = lo2;
#pragma unroll
  for (int i = 1; i < 4 * M; ++i) {
    const __nv_bfloat162 e = *reinterpret_cast<const __nv_bfloat162*>(&v[i]);
    lo2 = __hmin2_nan(lo2, e);
    hi2 = __hmax2_nan(hi2, e);
  }
#pragma unroll
  for (int off = 1; off < 4 / M; off <<= 1) {
    lo2 = __hmin2_nan(lo2, __shfl_xor_sync(lanes, lo2, off));
    hi2 = __hmax2_nan(hi2, __shfl_xor_sync(lanes, hi2, off));
  }
  *par = group_params(__bfloat162float(__hmin_nan(__low2bfloat16(lo2), __high2bfloat16(lo2))),
                      __bfloat162float(__hmax_nan(__low2bfloat16(hi2), __high2bfloat16(hi2))));
  const float s = param_scale(*par), m = param_min(*par);
#pragma unroll
  for (int j = 0; j < M; ++j) words[j] = 0u;
  if (!(s > 0.f)) return;                      // a constant group, or NaN
  const float r0 = __fdividef(1.f, s), r = __fmaf_rn(r0, __fmaf_rn(-s, r0, 1.f), r0);   // 1 / s within 2^-24
  const float2 s2 = make_float2(s, s), m2 = make_float2(m, m), r2 = make_float2(r, r);
  const float2 snap = make_float2(24.f, 24.f), back = make_float2(kIntBias - 24.f, kIntBias - 24.f);
  const float2 bias = make_float2(kIntBias, kIntBias);
  float far = 0.f;
#pragma unroll
  for (int j = 0; j < M; ++j) {
    float2 f[4];
    Elem<__nv_bfloat16>::unpack2(x[j], f);
    words[j] = 0u - 0x4b400000u * 0x11111111u;   // of the eight biases
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 d = sub2(f[i], m2);
      const float2 nb = add2(fma2(d, r2, snap), back);
      const float2 rem = fma2(sub2(bias, nb), s2, d);
      far = fmaxf(far, fmaxf(fabsf(rem.x), fabsf(rem.y)));
      words[j] += __float_as_uint(nb.x) << nibble_shift(2 * i);
      words[j] += __float_as_uint(nb.y) << nibble_shift(2 * i + 1);
    }
  }
  if (2.f * far <= s) return;
#pragma unroll
  for (int j = 0; j < M; ++j) {
    float f[8];
    Elem<__nv_bfloat16>::unpack(x[j], f);
    words[j] = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) words[j] |= (code_bits(__fsub_rn(f[i], m), s, r) & 15u) << nibble_shift(i);
  }
}

// ---- prefill -> cache hand-off ------------------------------------------------
struct PackParams {
  decode::PackParams d;
  long long blocks_per_b;
  int base[RATP_MAX_HEADS + 1];    // first block (within a batch item) of each head
};

// The last head h < H with base[h] <= at.
__device__ __forceinline__ int head_at(const int* base, int H, int at) {
  int lo = 0, hi = H - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (base[mid] <= at) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Dh/16 threads per row, kPackRows rows per thread; a block holds rows of one
// (b, h): its dilated rows first (quantised), then its ring rows (copied).
// Heads take blocks as they need (base[h]): a dense head has D times a dilated
// one's rows.  A thread has all its rows' loads in flight at once, and the
// block's index arithmetic and a group's parameters are spread over 16 channels.
// Bound by its reads and, close behind, by the arithmetic of the codes: 4 x 8192
// tokens of 2 dense heads and 30 of D = 4 (210 MB) take 42 us, 5 TB/s (with 8
// channels a thread 57.6 us, unpacked arithmetic 45 us).
constexpr int kPackRows = 2;
template <int DH>
__global__ void __launch_bounds__(256)
pack_kernel(const __grid_constant__ PackParams pp) {
  const decode::PackParams& p = pp.d;
  constexpr int TPR = DH / 16;
  constexpr int RPB = 256 / TPR;
  const int b = blockIdx.x / pp.base[p.H], at = blockIdx.x - b * pp.base[p.H];
  const int h = head_at(pp.base, p.H, at);
  const int r0 = (at - pp.base[h]) * (RPB * kPackRows) + threadIdx.x / TPR;
  const int li = threadIdx.x % TPR;
  const bool dense = decode::is_dense(p.dense_bits, h);
  const int Dd = dense ? 1 : p.D;
  const int n_dil = p.T / Dd;
  const int w_lo = max(0, p.T - p.W);
  const int n_ring = (p.W > 0) ? (p.T - w_lo) : 0;
  if (at == 0 && threadIdx.x == 0) p.len[b] = p.T;
  const long long src_base = (long long)b * p.T * p.H * DH + (long long)h * DH + li * 16;
  [[maybe_unused]] const long long n_src = (long long)p.B * p.T * p.H * DH;
  const long long block0 = (long long)b * pp.blocks_per_b + head_block(p.dense_bits, h, p.T_max, p.D);
  Block<DH>* const blocks = reinterpret_cast<Block<DH>*>(p.Kc) + block0;
  const unsigned lanes = 0x3u << ((threadIdx.x & 31) & ~1);

  uint4 in[kPackRows][2][2];
#pragma unroll
  for (int i = 0; i < kPackRows; ++i) {
    const int r = r0 + i * RPB;
    const int pos = r < n_dil ? r * Dd + Dd - 1 : w_lo + (r - n_dil);
    const long long src = src_base + (long long)pos * p.H * DH;
    const bool there = r < n_dil + n_ring && RATP_IN(src, 16, n_src);
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        in[i][s][j] = there ? __ldcs(reinterpret_cast<const uint4*>((s == 0 ? p.hk : p.hv) + src) + j)
                            : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int i = 0; i < kPackRows; ++i) {
    const int r = r0 + i * RPB;                // the same for a group's 2 lanes
    if (r < n_dil) {
      if (!RATP_IN(block0 + r / kStep, 1, p.B * pp.blocks_per_b)) continue;
      Block<DH>& blk = blocks[r / kStep];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        uint32_t par, w[2];
        quantise<2>(in[i][s], w, &par, lanes);
        *reinterpret_cast<uint2*>(&(s == 0 ? blk.k : blk.v)[r % kStep][2 * li]) = make_uint2(w[0], w[1]);
        if ((li & 1) == 0) (s == 0 ? blk.kp : blk.vp)[r % kStep][li / 2] = par;
      }
    } else if (r < n_dil + n_ring) {
      const long long dst = (((long long)b * p.H + h) * p.W + (w_lo + (r - n_dil)) % p.W) * DH + li * 16;
      if (!RATP_IN(dst, 16, (long long)p.B * p.H * p.W * DH)) continue;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        reinterpret_cast<uint4*>(p.Kw + dst)[j] = in[i][0][j];
        reinterpret_cast<uint4*>(p.Vw + dst)[j] = in[i][1][j];
      }
    }
  }
}

// ---- read-back: the values that the held rows stand for, fp32 ------------------
// A CTA reads one block of slots; a thread has quads of 4 channels, 256 apart, so
// that every store of a warp is 512 contiguous bytes.  Bound by its writes (8 times
// the codes): 311 000 rows of 128 channels take 31 us, 5.8 TB/s.
struct ReadParams {
  const void* blocks;
  float* out;                      // [B][rows_per_b][Dh]
  long long rows_per_b;
  int B, H, D, T_max, value;       // value: 0 the keys, 1 the values
  int base[RATP_MAX_HEADS + 1];    // first block (within a batch item) of each head
  unsigned long long dense_bits[RATP_MAX_HEADS / 64];
};
template <int DH>
__global__ void __launch_bounds__(256)
unpack_kernel(const __grid_constant__ ReadParams p) {
  constexpr int QPR = DH / 4, N = kStep * QPR / 256;     // quads per row, per thread
  const int b = blockIdx.x / p.base[p.H], at = blockIdx.x - b * p.base[p.H];
  const int h = head_at(p.base, p.H, at);
  const int cap = decode::is_dense(p.dense_bits, h) ? p.T_max : p.T_max / p.D;
  const int r0 = (at - p.base[h]) * kStep;
  const Block<DH>& blk = static_cast<const Block<DH>*>(p.blocks)[blockIdx.x];
  const uint32_t* codes = p.value ? &blk.v[0][0] : &blk.k[0][0];
  const uint32_t* params = p.value ? &blk.vp[0][0] : &blk.kp[0][0];
  const long long row0 = (long long)b * p.rows_per_b + decode::head_offset(p.dense_bits, h, p.T_max, p.D) + r0;
  float4* out = reinterpret_cast<float4*>(p.out) + row0 * QPR;
  const int n = min(kStep, cap - r0) * QPR;              // the last block of a head may be partly slots it has not
  uint32_t w[N], par[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int q = threadIdx.x + 256 * j;
    w[j] = codes[q >> 1];
    par[j] = params[q >> 3];
  }
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int q = threadIdx.x + 256 * j;
    if (q >= n || !RATP_IN(row0 + q / QPR, 1, p.B * p.rows_per_b)) continue;
    const float s = param_scale(par[j]), m = param_min(par[j]);
    const uint32_t x = w[j] >> ((q & 1) * 8);  // channels 4, 5, 6, 7 are the nibbles 2, 6, 3, 7
    float f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __fadd_rn(m, __fmul_rn((float)((x >> nibble_shift(i)) & 15u), s));
    __stcs(out + q, make_float4(f[0], f[1], f[2], f[3]));
  }
}

// ---- decode -------------------------------------------------------------------
__device__ __forceinline__ void mma_bf16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Code pairs of a word as bf16 pairs kOffset + n (channels 2i, 2i + 1).
constexpr float kOffset = 16.f, kMiddle = 7.5f;
constexpr int kFold = 8;             // steps between two takings out of the offset: 256 keys of a warp
__device__ __forceinline__ uint32_t pair_of(uint32_t w, int i) {
  const uint32_t at = i == 0 ? w << 3 : w >> (4 * i - 3);
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(at), "r"(0x00780078u), "r"(0x41804180u));   // (a & b) | c
  return r;
}

template <int DH>
struct Lane {
  static constexpr int NW = DH / 32;           // K words per key and lane (a quarter of the channels)
  static constexpr int NV = DH / 64;           // V words per key and lane (an eighth)
};

// Copy to shared memory, completing on `bar`.  One thread; 16-byte multiples.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               :: "r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}

template <int N>
__device__ __forceinline__ void read_words(uint32_t* r, const uint32_t* src) {
  if constexpr (N == 4) {
    const uint4 x = *reinterpret_cast<const uint4*>(src);
    r[0] = x.x; r[1] = x.y; r[2] = x.z; r[3] = x.w;
  } else if constexpr (N == 2) {
    const uint2 x = *reinterpret_cast<const uint2*>(src);
    r[0] = x.x; r[1] = x.y;
  } else {
    r[0] = *src;
  }
}

// Running softmax of one warp.  m is the reference of the weights 2^(s - m):
// it follows the running maximum only when a score passes it by more than
// kSlack, so a weight is at most 2^kSlack and most steps rescale nothing.
constexpr float kSlack = 8.f;
template <int DH>
struct Acc {
  float m, l;              // l: this lane's share
  float zm, zo;            // this lane's column: fp32 sums of w (m + 7.5 s) and of the parts of w s still offset in c
  float c[DH / 16][4];     // MMA j: channels 2 of this lane's Dh/8 x columns
};

template <int DH, int N>
__device__ __forceinline__ void weigh(Acc<DH>& a, const float* s, float* p) {
  float top = s[0];
#pragma unroll
  for (int i = 1; i < N; ++i) top = fmaxf(top, s[i]);
  if (__any_sync(0xffffffffu, top > a.m + kSlack)) {       // always so at the first finite score (m = -inf)
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    const float m = fmaxf(a.m, top);
    const float r = exp2f(a.m - m);
    a.l *= r;
    a.zm *= r;
    a.zo *= r;
#pragma unroll
    for (int j = 0; j < DH / 16; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) a.c[j][i] *= r;
    a.m = m;
  }
  const float m = a.m == -INFINITY ? 0.f : a.m;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    p[i] = exp2f(s[i] - m);
    a.l += p[i];
  }
}

// B operand of the values: this lane's column of the weights x[0..3] of keys
// t, 4 + t, 8 + t, 12 + t.  rest = 0 (columns 0..3): their bf16 parts; rest =
// 1 (columns 4..7): the bf16 of what those leave.  sum: what was taken.
__device__ __forceinline__ void split_weights(const float* x, float rest, uint32_t* b, float* sum) {
  float got = 0.f;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t hi = pack_bf16x2(x[2 * i], x[2 * i + 1]);
    const float y0 = fmaf(-rest, __uint_as_float(hi << 16), x[2 * i]);
    const float y1 = fmaf(-rest, __uint_as_float(hi & 0xffff0000u), x[2 * i + 1]);
    b[i] = pack_bf16x2(y0, y1);
    got += __uint_as_float(b[i] << 16) + __uint_as_float(b[i] & 0xffff0000u);
  }
  *sum = got;
}

// Weights of keys t, 4 + t, 8 + t, 12 + t of a 16-key tile, whose lane (g, t)
// holds those of keys g (p0) and g + 8 (p1).
__device__ __forceinline__ void gather_weights(float p0, float p1, int t, float* pw) {
  pw[0] = __shfl_sync(0xffffffffu, p0, 4 * t);
  pw[1] = __shfl_sync(0xffffffffu, p0, 16 + 4 * t);
  pw[2] = __shfl_sync(0xffffffffu, p1, 4 * t);
  pw[3] = __shfl_sync(0xffffffffu, p1, 16 + 4 * t);
}

template <int DH>
__device__ __forceinline__ void attend_codes(Acc<DH>& a, const Block<DH>& st, const uint32_t (*qf)[2],
                                             const float* qsum, float scale_log2, int n, int g, int t) {
  constexpr int NW = Lane<DH>::NW, NV = Lane<DH>::NV, P = DH / kGroup;
  constexpr int R = kStep / 8;                 // keys g + 8 r of this lane
  float s[R], p[R];
#pragma unroll
  for (int u = 0; u < kStep / kTile; ++u) {
    uint32_t w0[NW], w1[NW];
    read_words<NW>(w0, &st.k[16 * u + g][t * NW]);
    read_words<NW>(w1, &st.k[16 * u + g + 8][t * NW]);
    float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 2 * NW; ++j) {         // 4 channels of each quarter per MMA
      const int w = j / 2, i = 2 * (j % 2);
      mma_bf16(d, pair_of(w0[w], i), pair_of(w1[w], i), pair_of(w0[w], i + 1), pair_of(w1[w], i + 1), qf[j][0], qf[j][1]);
    }
    // lanes t = 0, 1 hold quarters (0, 1) and (2, 3); the others' columns are
    // zero, and so are their qsum
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      uint32_t par[2];
      if constexpr (P == 4) read_words<2>(par, &st.kp[16 * u + g + 8 * r][2 * (t & 1)]);
      else par[0] = par[1] = st.kp[16 * u + g + 8 * r][t & 1];
      const float sa = param_scale(par[0]), sb = param_scale(par[1]);
      float x = fmaf(sa, fmaf(-kOffset, qsum[0], d[2 * r]), param_min(par[0]) * qsum[0]);
      x += fmaf(sb, fmaf(-kOffset, qsum[1], d[2 * r + 1]), param_min(par[1]) * qsum[1]);
      x += __shfl_xor_sync(0xffffffffu, x, 1);
      s[2 * u + r] = __shfl_sync(0xffffffffu, x, 0, 4) * scale_log2;
    }
  }
  if (n < kStep) {
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (8 * r + g >= n) s[r] = -INFINITY;
  }
  weigh<DH, R>(a, s, p);
  const float rest = g < 4 ? 0.f : 1.f;
#pragma unroll
  for (int u = 0; u < kStep / kTile; ++u) {
    float pw[4], x[4], got;
    gather_weights(p[2 * u], p[2 * u + 1], t, pw);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t par = st.vp[16 * u + 4 * j + t][(g & 3) * P / 4];
      x[j] = pw[j] * param_scale(par);
      a.zm = fmaf(pw[j], fmaf(kMiddle, param_scale(par), param_min(par)), a.zm);
    }
    uint32_t bw[2];
    split_weights(x, rest, bw, &got);
    a.zo += got;
    uint32_t v[4][NV];
#pragma unroll
    for (int j = 0; j < 4; ++j) read_words<NV>(v[j], &st.v[16 * u + 4 * j + t][g * NV]);
#pragma unroll
    for (int w = 0; w < NV; ++w) {
      // low halves: channels 0, 2, 4, 6 of the word; high halves: 1, 3, 5, 7
      const uint32_t l01 = __byte_perm(v[0][w], v[1][w], 0x5410), h01 = __byte_perm(v[0][w], v[1][w], 0x7632);
      const uint32_t l23 = __byte_perm(v[2][w], v[3][w], 0x5410), h23 = __byte_perm(v[2][w], v[3][w], 0x7632);
#pragma unroll
      for (int i = 0; i < 4; ++i)              // channels 2i (row g) and 2i + 1 (row g + 8)
        mma_bf16(a.c[4 * w + i], pair_of(l01, i), pair_of(h01, i), pair_of(l23, i), pair_of(h23, i), bw[0], bw[1]);
    }
  }
}

// Takes the offset of the codes multiplied so far out of the values' sums.
template <int DH>
__device__ __forceinline__ void take_offset(Acc<DH>& a, int t) {
  float z = a.zo;                              // of column g, over this lane's keys
  z += __shfl_xor_sync(0xffffffffu, z, 1);
  z += __shfl_xor_sync(0xffffffffu, z, 2);
  const float z0 = __shfl_sync(0xffffffffu, z, 8 * t), z1 = __shfl_sync(0xffffffffu, z, 8 * t + 4);   // columns 2t, 2t + 1
#pragma unroll
  for (int j = 0; j < DH / 16; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) a.c[j][i] = fmaf(-(kOffset + kMiddle), i & 1 ? z1 : z0, a.c[j][i]);
  a.zo = 0.f;
}

// ---- ring rows: bf16, kRingStep of them in a stage ------------------------------
// One copy a row, into rows 16 bytes apart from a multiple of the banks, which
// leaves the lanes' reads two to a bank.
template <int DH>
struct RingStage {
  uint4 k[kRingStep][DH / 8 + 1];
  uint4 v[kRingStep][DH / 8 + 1];
};

// n <= kRingStep ring rows from ring row `first` on (wrapping at W) into a
// stage, by the warp.
template <int DH>
__device__ __forceinline__ void fetch_ring(uint32_t stage, const __nv_bfloat16* kw, const __nv_bfloat16* vw, int first,
                                           int W, int n, int lane, uint32_t bar) {
  constexpr uint32_t kRow = DH * 2;
  static_assert(kRingStep == 8, "lanes 0..7 K, 8..15 V");
  if (lane == 0) sm100::mbar_arrive_expect_tx(bar, 2u * kRow * (uint32_t)n);
  __syncwarp();
  const int r = lane & 7;
  if (lane < 16 && r < n) {
    const int row = first + r < W ? first + r : first + r - W;
    const uint32_t dst = stage + (uint32_t)r * (kRow + 16) + (lane < 8 ? 0u : (uint32_t)offsetof(RingStage<DH>, v));
    bulk_load(dst, (lane < 8 ? kw : vw) + (long long)row * DH, kRow, bar);
  }
}

// As attend_codes, with half an MMA tile's keys.
template <int DH>
__device__ __forceinline__ void attend_ring(Acc<DH>& a, const RingStage<DH>& st, const uint32_t (*qf)[2],
                                            float scale_log2, int n, int g, int t) {
  constexpr int NW = Lane<DH>::NW, NV = Lane<DH>::NV;
  static_assert(kRingStep == 8, "keys g of the lanes");
  float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    const uint4 k = st.k[g][t * NW + w];
    mma_bf16(d, k.x, 0u, k.y, 0u, qf[2 * w][0], qf[2 * w][1]);
    mma_bf16(d, k.z, 0u, k.w, 0u, qf[2 * w + 1][0], qf[2 * w + 1][1]);
  }
  float s = d[0] + d[1], p, pw[4], got;
  s += __shfl_xor_sync(0xffffffffu, s, 1);
  s = __shfl_sync(0xffffffffu, s, 0, 4) * scale_log2;
  if (g >= n) s = -INFINITY;
  weigh<DH, 1>(a, &s, &p);
  gather_weights(p, 0.f, t, pw);
  uint32_t bw[2];
  split_weights(pw, g < 4 ? 0.f : 1.f, bw, &got);
#pragma unroll
  for (int w = 0; w < NV; ++w) {
    const uint4 v0 = st.v[t][g * NV + w], v1 = st.v[4 + t][g * NV + w];
    const uint32_t x[4] = {v0.x, v0.y, v0.z, v0.w}, y[4] = {v1.x, v1.y, v1.z, v1.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      mma_bf16(a.c[4 * w + i], __byte_perm(x[i], y[i], 0x5410), __byte_perm(x[i], y[i], 0x7632), 0u, 0u, bw[0], bw[1]);
  }
}

static_assert(sizeof(RingStage<128>) <= sizeof(Block<128>) && sizeof(RingStage<64>) <= sizeof(Block<64>), "stage");

template <int DH>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
decode_kernel(const Params pp) {
  const decode::Params& p = pp.d;
  constexpr int W8 = DH / 8;
  constexpr int NQ = DH / 16;                  // score MMAs per tile
  constexpr int NE = kWarps + 1;               // merged entries: the warps and the query's own key

  __shared__ __align__(16) float s_self[2][DH];
  __shared__ float s_m[NE], s_l[NE];
  __shared__ __align__(16) float s_acc[NE][DH];
  __shared__ int s_last;
  __shared__ __align__(8) unsigned long long s_bar[kWarps][kStages];
  __shared__ int s_abort;
  extern __shared__ __align__(128) uint8_t s_stages[];   // Block<DH>[kWarps][kStages]

  const int b = blockIdx.x / p.splits_per_b;
  const int rem = blockIdx.x - b * p.splits_per_b;
  const int h = decode::head_of_split(p, rem);
  const int split = rem - p.split_base[h];
  const int tid = threadIdx.x;
  const bool dense = decode::is_dense(p.dense_bits, h);
  const int cap = dense ? p.T_max : p.T_max / p.D;
  const long long block0 = (long long)b * pp.blocks_per_b + head_block(p.dense_bits, h, p.T_max, p.D);
  [[maybe_unused]] const long long n_blocks = (long long)p.B * pp.blocks_per_b;
  Block<DH>* const blocks = reinterpret_cast<Block<DH>*>(p.Kc) + block0;

  // as in decode.cuh: let the next step be scheduled, warm L2 with this
  // split's first rows, then wait for the kernels before this one
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == 0) {
    const long long first = (long long)split * p.split_keys / kStep;
    const long long n = min((long long)kPrefetchBlocks, blocks_of(cap) - first);
    if (n > 0 && RATP_IN(block0 + first, n, n_blocks))
      decode::bulk_prefetch_l2(blocks + first, (uint32_t)(n * sizeof(Block<DH>)));
    s_abort = 0;
#pragma unroll
    for (int i = 0; i < kWarps * kStages; ++i) sm100::mbar_init(sm100::smem_u32(&s_bar[0][0] + i), 1);
    sm100::fence_barrier_init();
  }
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int t = p.len[b];
  // the query and the recurrence's inputs: on their way with the length, ahead
  // of the cache stream
  const long long bh = (long long)b * p.H + h;
  [[maybe_unused]] const long long n_tok = (long long)p.B * p.H * DH;
  const int warp = tid >> 5, lane = tid & 31, g = lane >> 2, tq = lane & 3;
  const bool q_ok = RATP_IN(bh * DH, DH, n_tok);
  uint4 qv[DH / 32];                           // this lane's quarter of the channels
#pragma unroll
  for (int i = 0; i < DH / 32; ++i)
    qv[i] = q_ok ? reinterpret_cast<const uint4*>(p.q + bh * DH + tq * (DH / 4))[i] : make_uint4(0u, 0u, 0u, 0u);
  constexpr int kIn = 2 * DH / kThreads;
  decode::StepInput in[kIn];
  if (split == 0 && q_ok) {
#pragma unroll
    for (int i = 0; i < kIn; ++i) in[i] = decode::load_input(p, bh, (tid + i * kThreads) / DH, (tid + i * kThreads) % DH, DH);
  }
  const int Dd = dense ? 1 : p.D;
  bool active = true;
  int n_slots = 0, w_lo = 0, n_win = 0, n_used = 1, app_slot = 0;
  if ((unsigned)t >= (unsigned)p.T_max) {      // full, or a length that is none
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
    [[maybe_unused]] const long long n_ring = (long long)p.B * p.H * p.W * DH;
    // ---- this split's share: units [u0, u1) of slots, then of ring keys ----
    const long long u0 = (long long)split * p.split_keys, u1 = u0 + p.split_keys;
    const int s_end = (int)min((long long)n_slots, u1);
    const auto ring_at = [&](long long u) {
      return (int)min((long long)n_win, (max(u - n_slots, 0ll) + kRingUnits - 1) / kRingUnits);
    };
    const int k0 = (int)min((long long)n_slots, u0) + warp * kStep;      // u0 is whole blocks
    Block<DH>* const stages = reinterpret_cast<Block<DH>*>(s_stages) + warp * kStages;
    const uint32_t stage0 = sm100::smem_u32(stages), bar0 = sm100::smem_u32(&s_bar[warp][0]);
    // a warp's steps: rows k0 + i kRows .. of the cache, then its share of the ring
    constexpr int kRows = kWarps * kStep;
    const int r_begin = ring_at(u0), r_end = RATP_IN(bh * p.W * DH, (long long)p.W * DH, n_ring) ? ring_at(u1) : 0;
    const __nv_bfloat16* kw = p.Kw + bh * p.W * DH;
    const __nv_bfloat16* vw = p.Vw + bh * p.W * DH;
    int at = k0, fill = 0;                     // next cached rows to fetch, and the stage for them
    int ring = r_begin + warp * kRingStep;     // next ring rows, after the cached ones, and where they lie
    int ring_row = n_win > 0 ? (w_lo + ring) % p.W : 0;
    const int ring_hop = n_win > 0 ? kWarps * kRingStep % p.W : 0;
    auto fetch_next = [&]() {
      const uint32_t stage = stage0 + fill * (uint32_t)sizeof(Block<DH>);
      if (at < s_end) {
        if (lane == 0 && RATP_IN(block0 + at / kStep, 1, n_blocks)) {
          sm100::mbar_arrive_expect_tx(bar0 + 8 * fill, (uint32_t)sizeof(Block<DH>));
          bulk_load(stage, blocks + at / kStep, (uint32_t)sizeof(Block<DH>), bar0 + 8 * fill);
        }
        at += kRows;
      } else if (ring < r_end) {
        fetch_ring<DH>(stage, kw, vw, ring_row, p.W, min(kRingStep, r_end - ring), lane, bar0 + 8 * fill);
        ring += kWarps * kRingStep;
        ring_row += ring_hop;
        ring_row = ring_row < p.W ? ring_row : ring_row - p.W;
      }
      fill = fill + 1 == kStages ? 0 : fill + 1;
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch_next();

    // ---- the recurrence, the appended row (the first cached rows are on their way) ----
    if (split == 0) {
      decode::recurrence_step<DH, kThreads>(p, bh, t, s_self[0], s_self[1], q_ok ? in : nullptr, [](int, int, __nv_bfloat16) {});
      if (t % Dd == Dd - 1) {
        if (app_slot >= cap) {
          if (tid == 0) raise_error(RATP_ERR_CAPACITY);
        } else if (tid < 2 * W8 && RATP_IN(block0 + app_slot / kStep, 1, n_blocks)) {
          // 8 channels per thread; W8 threads per stream, in whole groups of 4
          const int st = tid / W8, w = tid % W8;
          uint32_t par;
          float2 f[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) f[i] = *reinterpret_cast<const float2*>(&s_self[st][8 * w + 2 * i]);
          const uint4 x = Elem<__nv_bfloat16>::pack2(f);
          uint32_t code;
          quantise<1>(&x, &code, &par, 0xfu << (lane & ~3));
          Block<DH>& blk = blocks[app_slot / kStep];
          (st == 0 ? blk.k : blk.v)[app_slot % kStep][w] = code;
          if ((w & 3) == 0) (st == 0 ? blk.kp : blk.vp)[app_slot % kStep][w / 4] = par;
        }
      }
    }

    uint32_t qf[NQ][2];
    float qsum[2];
    {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < DH / 32; ++i) {
        float f[8];
        Elem<__nv_bfloat16>::unpack(qv[i], f);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum += f[j];
        const bool mine = g == tq;             // B's column n = g is quarter n alone
        qf[2 * i][0] = mine ? qv[i].x : 0u;
        qf[2 * i][1] = mine ? qv[i].y : 0u;
        qf[2 * i + 1][0] = mine ? qv[i].z : 0u;
        qf[2 * i + 1][1] = mine ? qv[i].w : 0u;
      }
      qsum[0] = __shfl_sync(0xffffffffu, sum, 2 * tq, 4);          // quarters 2t, 2t + 1
      qsum[1] = __shfl_sync(0xffffffffu, sum, 2 * tq + 1, 4);
      if (tq >= 2) qsum[0] = qsum[1] = 0.f;
    }

    Acc<DH> a;
    a.m = -INFINITY;
    a.l = 0.f;
    a.zm = a.zo = 0.f;
#pragma unroll
    for (int j = 0; j < NQ; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) a.c[j][i] = 0.f;

    int use = 0;
    uint32_t phase = 0;                        // of the barrier of stage `use`
    auto landed = [&]() { return sm100::warp_all(sm100::mbar_wait(bar0 + 8 * use, phase, &s_abort)); };
    auto next = [&]() {
      __syncwarp();
      use = use + 1 == kStages ? 0 : use + 1;
      phase ^= use == 0 ? 1u : 0u;
    };
    int k = k0, r = r_begin + warp * kRingStep;
    int folded = 0;                            // steps since the offset was taken out
    for (; k < s_end; k += kRows) {
      fetch_next();
      if (!landed()) break;
      if (s_end - k < kStep) {                 // rows past the last slot hold anything: 0 times their step must be 0
        uint32_t* par = &stages[use].vp[0][0];
        for (int i = (s_end - k) * (DH / kGroup) + lane; i < kStep * (DH / kGroup); i += 32) par[i] = 0u;
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
      }
      attend_codes<DH>(a, stages[use], qf, qsum, p.scale_log2, s_end - k, g, tq);
      if (++folded == kFold) {
        take_offset<DH>(a, tq);
        folded = 0;
      }
      next();
    }
    for (; k >= s_end && r < r_end; r += kWarps * kRingStep) {
      fetch_next();
      if (!landed()) break;
      RingStage<DH>& st = reinterpret_cast<RingStage<DH>&>(stages[use]);
      if (r_end - r < kRingStep) {             // likewise the values past the last row
        uint4* v = &st.v[0][0];
        for (int i = (r_end - r) * (DH / 8 + 1) + lane; i < kRingStep * (DH / 8 + 1); i += 32) v[i] = make_uint4(0u, 0u, 0u, 0u);
        __syncwarp();
      }
      attend_ring<DH>(a, st, qf, p.scale_log2, min(kRingStep, r_end - r), g, tq);
      next();
    }
    // given up: every copy under way lands before the CTA ends
    for (int i = 0; i < kStages && (k < s_end || r < r_end); ++i) {
      sm100::mbar_drain(bar0 + 8 * use, phase);
      next();
      if (k < s_end) k += kRows; else r += kWarps * kRingStep;
    }

    // ---- this warp's entry ----
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) a.l += __shfl_xor_sync(0xffffffffu, a.l, off);
    // middles count once (columns 0..3); the offsets of both parts
    float z = fmaf(-(kOffset + kMiddle), a.zo, g < 4 ? a.zm : 0.f);
    z += __shfl_xor_sync(0xffffffffu, z, 1);
    z += __shfl_xor_sync(0xffffffffu, z, 2);
    z += __shfl_xor_sync(0xffffffffu, z, 16);                      // lanes g and g + 4: quarter g % 4
    z = __shfl_sync(0xffffffffu, z, (g >> 1) << 2);                // of the quarter this lane's channels lie in
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
    decode::merge_entries<DH, NE, kThreads>(p, bh, split, n_used, s_m, s_l, s_acc, &s_last);
  }

  decode::advance_len(p, b);
}

}  // namespace decode_q4
}  // namespace ratp
