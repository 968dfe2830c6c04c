// linear_attn.cuh -- linear attention with a decay for each head: the mixer
// whose state has a fixed size (a layer of a stack may use it in place of the
// dilated attention and its cache).
//
//   S_t = a S_{t-1} + k_t v_t^T,  o_t = scale q_t S_t,   a = exp(log_decay[h])
//
// S is Dh x Dh per (b, h), fp32.  Two kernels:
//
// * recurrent_kernel walks the tokens one by one (a decode token, or a piece
//   of at most kRecurrentTokens): the state is read and written once, which is
//   all its time (64 x 16 states of 128 x 128, 134 MB: 20 us in a row, 24 us with
//   cold caches, 6.7 and 5.6 TB/s).
// * chunk_kernel takes 128 tokens at a time on the tensor cores.  With S the
//   state before the chunk, n the tokens in it, i, j = 0 .. n-1:
//     o_i  = scale a^{i+1} q_i S + sum_{j <= i} scale a^{i-j} (q_i . k_j) v_j
//     S'   = a^n S + sum_j a^{n-1-j} k_j v_j^T
//   that is, with P = mask(Q K^T) * scale a^{i-j}: two products read against the
//   chunk's values and state, and one that advances the state.
//   No power of a is ever inverted, so any decay in (0, 1] is as exact as any
//   other.  P and the state enter their products rounded to bf16 (as the
//   attention's P does: the output is bf16 itself).  The state's own update
//   keeps all 24 bits of a^{n-1-j} k_j as three bf16 terms (three products),
//   the products accumulate one chunk only, and the running state is fp32 in
//   registers, so the state that is handed on is as good as fp32 sums (two
//   terms, 16 bits, left it 10 times further off than the plain fp32 form).
//
// A sequence is a chain over its chunks, so few (b, h) leave SMs idle: then
// the chunks are cut into segments.  chunk_kernel<DH, false> computes every
// segment's own state (from zero), combine_kernel turns those into the state
// before each segment, and chunk_kernel<DH, true> runs all segments at once.  The
// three are programmatic dependents: each starts beside the end of the one before
// and waits for it where it reads a state.
//
// Roles of chunk_kernel (448 threads, one CTA per SM):
//   warps 0-3   P: read Q K^T from TMEM, mask, decay, write bf16 P to TMEM over
//               it; then o = scale a^{i+1} O1 + O2 out of TMEM to memory;
//   warps 4-11  state, half of its columns to each four warps: scale K in place
//               to the first term, the others beside it, 32 tokens at a time
//               through two buffers; S = a^n S + (TMEM) in registers; S as bf16
//               in shared memory;
//   warp 12     TMA producer: Q, K, V tiles through a ring of kSlots tiles;
//   warp 13     TMEM and the MMA issuer: P = Q K^T (M 128 tokens, N 128 tokens),
//               O1 = Q S, O2 = P V, SL = K'^T V (M = Dh).  Q K^T of the next
//               chunk goes between the first and the other parts of SL, so that
//               P of the next chunk is worked out while this one's state is.
//   Without an output (<DH, false>) only SL is computed, in two buffers, and
//   warps 0-3 share the scaling of K.
// P V multiplies the values of the tokens after i by zeros, so a value that is not
// finite would reach the outputs of its chunk before it.  It also stays in the
// state, so one look at the last chunk's o tells whether a CTA met any; if so, it
// does its chunks over in a pass that takes such values out of V once the state's
// products have read them (4 x 8192 x 32 x 128: 240 us; with V scanned in every
// pass, by two more warps, 306 us).
// Bound: the 4 tiles of memory traffic per chunk and (b, h) are the floor (six
// products take less), but a chunk is a chain: S as bf16, Q S, then P V and o, and
// beside it the scaling of K, its products and S.  One CTA has all of an SM's TMEM
// and shared memory, so little else hides the chain's latencies: 3.6 us a chunk,
// 1.4 times its share of the memory's time.  4 x 8192 x 32 x 128 (128 CTAs): 240 us
// of 165, and 284 us in a run of a second, whose clock the power limit holds at 1.5
// GHz; 2 x 16384 x 16 x 128 (four segments, K and V read twice): 196 and 217 us of
// 82.  Scaling that ran a chunk ahead, with six slots, took 268 to 292 us in place of
// 246 for the first.  For Dh = 64 the chain is nearly as long on half the bytes:
// 4 x 8192 x 32 x 64 in 167 us (176 in a run) of 82.  At 128 registers chunk_kernel<128, true> spills
// 48 bytes and loads 52 a thread, <64, true> 32 and 68 (the repair pass 80 and 168).
#pragma once
#include "sm100.cuh"

namespace ratp {
namespace linear_attn {

constexpr int C = 128;                 // tokens per chunk
constexpr int kThreads = 448;
constexpr int kStateWarps = 8;         // warps 4 .. 11
constexpr int kProducerWarp = 12;
constexpr int kMmaWarp = 13;
constexpr int kSlots = 5;
constexpr int kPart = 32;               // tokens whose scaled K is handed to the MMA at a time
constexpr int kParts = C / kPart;
// Sequences of up to this many tokens run token by token.  Measured, us (token by
// token / in chunks, states in and out), T = 8, 16, 32:
//   Dh 128,    4 (b, h):  7.7 / 13.5,  13.3 / 13.5,  24.1 / 13.7
//   Dh 128, 1024 (b, h): 45.9 / 87.9,  81.7 / 88.3, 158.4 / 90.3
//   Dh  64,    4 (b, h):  6.1 /  7.8,  10.4 /  7.8,  18.7 /  7.7
//   Dh  64, 1024 (b, h): 16.4 / 52.8,  28.8 / 52.8,  53.5 / 52.9
constexpr int kRecurrentTokens = 16;

// a^n for n >= 0 tokens.  log_decay is clamped to a finite value, below which
// every power but the 0th is zero in fp32 (a NaN stays one).
__device__ __forceinline__ double exact_power(float log_decay, double n) {
  return n == 0.0 ? 1.0 : exp((log_decay < -1.0e4f ? -1.0e4 : (double)log_decay) * n);
}
__device__ __forceinline__ float decay_power(float log_decay, double n) { return (float)exact_power(log_decay, n); }

// The same to twice the bits, for what a state is multiplied by again and again:
// a rounding of the power alone would drift the state by as many of its roundings
// as there are segments or tokens within the decay's reach (the chunks of a
// segment spread the low part over their powers, see update).
// An infinite state stays what it is: the low part, which may be negative or zero,
// is multiplied by the largest finite number in its place.
struct Decay {
  float hi, lo;
  __device__ __forceinline__ float step(float s, float add) const {
    constexpr float kMost = 3.402823466e38f;
    return fmaf(hi, s, fmaf(lo, fminf(fmaxf(s, -kMost), kMost), add));
  }
};
__device__ __forceinline__ Decay decay_pair(float log_decay, double n) {
  const double x = exact_power(log_decay, n);
  const float hi = (float)x;
  return {hi, (float)(x - (double)hi)};
}

template <int DH>
struct Layout {
  static constexpr uint32_t kHalf = C * 128;             // 128 rows x 64 bf16
  static constexpr uint32_t kTile = (DH / 64) * kHalf;
  static constexpr uint32_t kOffO = kSlots * kTile;      // o of a chunk on its way out
  static constexpr uint32_t kOffS = kOffO + kTile;       // S, bf16 [DH / 64][DH rows][64]
  static constexpr uint32_t kSHalf = DH * 128;
  static constexpr uint32_t kOffPow = kOffS + (DH / 64) * kSHalf;    // a^0 .. a^128
  static constexpr uint32_t kOffDecay = kOffPow + (C + 2) * 4;       // of a whole chunk, of the sequence's last
  static constexpr uint32_t kOffBar = kOffDecay + 2 * sizeof(Decay);
  static constexpr int kBars = 2 * kSlots + 15;                      // of a pass; there are two
  static constexpr uint32_t kOffCtl = kOffBar + 2 * kBars * 8;       // TMEM address, abort flag
  static constexpr uint32_t kOffFirst = kOffCtl + 16;                // first[DH], bytes
  // one CTA per SM whatever DH, since each takes all of TMEM
  static constexpr uint32_t kUsed = kOffFirst + DH + 1024;
  static constexpr uint32_t kBytes = kUsed > 120 * 1024 ? kUsed : 120 * 1024;
};
static_assert(Layout<128>::kBytes <= 232448, "shared memory of one CTA");

constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColP = 0;          // 128 columns: Q K^T, then P as bf16 pairs in the first 64
constexpr uint32_t kColO = 128;        // DH columns: Q S, scaled, += P V
constexpr uint32_t kColS = 256;        // DH columns: the state's products (with <DH, false> at 0 and 128)
constexpr uint32_t kColK = 384;        // 2 buffers x 3 terms x 16 columns: scaled K^T of 32 tokens
constexpr uint32_t kTermCols = kPart / 2;
constexpr uint32_t kBufCols = 3 * kTermCols;

struct Params {
  const float* log_decay;              // [H]
  const float* init;                   // [B][H][DH][DH] or NULL: the state before the sequence
  float* fin;                          // [B][H][DH][DH] or NULL: the state after it
  float* ws;                           // [B * H][n_seg][DH][DH]: segment states
  int B, T, H;
  int n_chunks, seg_chunks, n_seg;
  float scale;
};

// x * w of two floats as three bf16 terms each, which are its fp32 value's upper,
// middle and lower 8 bits (cut off, not rounded, so that every remainder is
// exact and the third term leaves nothing).
__device__ __forceinline__ void split3(float2 x, float2 w, uint32_t* t0, uint32_t* t1, uint32_t* t2) {
  auto upper = [](float2 v) { return __byte_perm(__float_as_uint(v.x), __float_as_uint(v.y), 0x7632); };
  auto cut = [](float2 v) {
    return make_float2(__uint_as_float(__float_as_uint(v.x) & 0xffff0000u), __uint_as_float(__float_as_uint(v.y) & 0xffff0000u));
  };
  const float2 y = mul2(x, w);
  *t0 = upper(y);
  const float2 r = sub2(y, cut(y));
  *t1 = upper(r);
  *t2 = upper(sub2(r, cut(r)));
}

// Named barrier `id` of `count` threads; true where every one of them passed true.
__device__ __forceinline__ bool group_all(int id, int count, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r) : "r"((uint32_t)ok), "r"(id), "r"(count) : "memory");
  return r != 0;
}

// One pass over a CTA's chunks.  REPAIR: the pass that does them over, with the
// values that are not finite taken out of P V.  Returns whether that is needed.
template <int DH, bool OUT, bool REPAIR>
__device__ __forceinline__ bool chunk_pass(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                           const CUtensorMap& tm_o, const Params& p, uint8_t* smem, uint32_t tmem) {
  using namespace sm100;
  using L = Layout<DH>;
  constexpr int NH = DH / 64;                            // 64-channel halves
  constexpr int kUnits = OUT ? 3 : 2;                    // tiles per chunk: (Q,) K, V
  constexpr int kK = OUT ? 1 : 0;                        // K's place among them
  const uint32_t sb = smem_u32(smem);
  const uint32_t bar0 = sb + L::kOffBar + (REPAIR ? L::kBars * 8u : 0u);
  const uint32_t b_full = bar0, b_empty = bar0 + 8 * kSlots;
  const uint32_t b_qk = bar0 + 8 * (2 * kSlots), b_p = b_qk + 8, b_o = b_qk + 16, b_ofree = b_qk + 24;
  // part g = kParts c + part of this CTA's tokens uses buffer g & 1, and these
  // barriers' phase g / 2
  const uint32_t b_kp = b_qk + 32;                       // [2]: part scaled
  const uint32_t b_kv = b_qk + 48;                       // [2]: its products done
  const uint32_t b_s = b_qk + 64, b_final = b_qk + 72;
  // chunk c's state products done, and (<DH, false>) their TMEM buffer read:
  // barriers [c & 1], phase c / 2
  const uint32_t b_pd = b_qk + 80, b_sf = b_qk + 96;
  const uint32_t b_qs = b_qk + 112;                      // Q S done
  float* s_pow = reinterpret_cast<float*>(smem + L::kOffPow);
  Decay* s_decay = reinterpret_cast<Decay*>(smem + L::kOffDecay);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + L::kOffCtl + 4);
  [[maybe_unused]] uint8_t* s_first = smem + L::kOffFirst;           // column x of V is not finite from token s_first[x] on
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // warp: known uniform

  // segment `seg` of (b, h)
  const int per = OUT ? p.n_seg : p.n_seg - 1;
  const int pair = blockIdx.x / per, seg = blockIdx.x - pair * per;
  const int b = pair / p.H, h = pair - b * p.H;
  const int c0 = seg * p.seg_chunks;
  const int n = min(p.seg_chunks, p.n_chunks - c0);      // chunks here
  const bool last_seg = seg == p.n_seg - 1;
  // the state after the last chunk is wanted by <DH, false> and by p.fin
  const bool want_end = !OUT || (last_seg && p.fin != nullptr);
  const int n_state = want_end ? n : n - 1;              // chunks whose state update is computed
  // tokens of chunk c (of this segment)
  auto tokens = [&](int c) { return min(C, p.T - (c0 + c) * C); };

  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(b_full + 8 * i, 1);
      mbar_init(b_empty + 8 * i, 1);
    }
    mbar_init(b_qk, 1);
    mbar_init(b_qs, 1);
    mbar_init(b_p, 128);
    mbar_init(b_o, 1);
    mbar_init(b_ofree, 128);
    for (int i = 0; i < 2; ++i) {
      mbar_init(b_kp + 8 * i, 128);
      mbar_init(b_kv + 8 * i, 1);
      mbar_init(b_pd + 8 * i, 1);
      mbar_init(b_sf + 8 * i, 32 * kStateWarps);
    }
    mbar_init(b_s, 32 * kStateWarps);
    mbar_init(b_final, 1);
    fence_barrier_init();
  }
  const float ld = p.log_decay[h];
  __syncthreads();
  bool again = false;                                    // known to warp 0 and the state warps
  // tile u of this CTA (chunk u / kUnits; (Q,) K, V in turn) lies in slot u % kSlots
  auto full_wait = [&](int u) { return mbar_wait(b_full + 8 * (u % kSlots), (uint32_t)(u / kSlots) & 1u, s_abort); };
  auto tile = [&](int u) { return sb + (uint32_t)(u % kSlots) * L::kTile; };

  auto kv_wait = [&](int g) { return mbar_wait(b_kv + 8 * (g & 1), (uint32_t)(g >> 1) & 1u, s_abort); };
  // a^{n-1-j} k_j, transposed, into TMEM (lane = channel, two tokens a column)
  // as three bf16 terms, for parts first, first + step, .. of chunk c by a
  // group of four warps: each takes the 32 channels of its TMEM lanes, 16 at a
  // time, straight from K's tile by transposing loads.  A part's buffer is free
  // once the products of the part before the last are done.
  auto scale_k = [&](int c, int first, int step) -> bool {
    const int m = tokens(c), quad = warp & 3, pair = lane & 3;
    const uint32_t t = tile(c * kUnits + kK) + (uint32_t)(quad >> 1) * L::kHalf;
    // this lane's row of the four 8 x 8 tiles (token, 16-byte chunk) of a load
    const int row = (lane >> 4) * 8 + (lane & 7), ch = (quad & 1) * 4 + ((lane >> 3) & 1);
#pragma unroll 1
    for (int part = first; part < kParts; part += step) {
      const int g = c * kParts + part;
      // everything is loaded before the buffer is waited for
      const bool mine = 32 * quad < DH;
      uint32_t raw[16];
      float2 w[4];                             // weights of tokens 8 i + 2 pair, + 1
      if (mine) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {          // tokens 16 x .. of the part
          const int tok = part * kPart + 16 * x + row;
#pragma unroll
          for (int lh = 0; lh < 2; ++lh)       // channels 16 lh .. of this warp's 32
            ldmatrix_x4_trans(t + (uint32_t)tok * 128 + (uint32_t)(((ch + 2 * lh) ^ (tok & 7)) * 16), raw + 8 * x + 4 * lh);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = m - 1 - (part * kPart + 8 * i + 2 * pair);
          w[i] = make_float2(s_pow[max(e, 0)], s_pow[max(e - 1, 0)]);       // tokens past the sequence are zero
        }
      }
      if (g >= 2 && !warp_all(kv_wait(g - 2))) return false;
      tc_fence_after();
      if (mine) {
        const uint32_t dst = tmem + ((uint32_t)(quad * 32) << 16) + kColK + (uint32_t)(g & 1) * kBufCols;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
#pragma unroll
          for (int lh = 0; lh < 2; ++lh) {
            uint32_t t0[4], t1[4], t2[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {      // register y: tokens 8 (y / 2) + 2 pair, + 1
              const uint32_t v = raw[8 * x + 4 * lh + y];
              split3(make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u)), w[2 * x + y / 2], &t0[y],
                     &t1[y], &t2[y]);
            }
            const uint32_t d = dst + ((uint32_t)(16 * lh) << 16) + 8 * x;
            tmem_st_16x128b_x2(d, t0);
            tmem_st_16x128b_x2(d + kTermCols, t1);
            tmem_st_16x128b_x2(d + 2 * kTermCols, t2);
          }
        }
        tmem_wait_st();
      }
      tc_fence_before();
      mbar_arrive(b_kp + 8 * (g & 1));
    }
    return true;
  };

  if (warp == kProducerWarp) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      prefetch_tmap(&tm_k);
      prefetch_tmap(&tm_v);
      if (OUT) prefetch_tmap(&tm_q);
      int u = 0;
      bool ok = true;
      for (int c = 0; c < n && ok; ++c) {
        const int t0 = (c0 + c) * C;
#pragma unroll
        for (int i = 0; i < kUnits; ++i, ++u) {
          const CUtensorMap* m = i == kK ? &tm_k : i == kK + 1 ? &tm_v : &tm_q;
          if (u >= kSlots && !mbar_wait(b_empty + 8 * (u % kSlots), (uint32_t)(u / kSlots - 1) & 1u, s_abort)) {
            ok = false;
            break;
          }
          const uint32_t fb = b_full + 8 * (u % kSlots);
          mbar_arrive_expect_tx(fb, L::kTile);
#pragma unroll
          for (int hf = 0; hf < NH; ++hf) tma_load_4d(tile(u) + hf * L::kHalf, m, fb, 64 * hf, h, t0, b);
        }
      }
      // every copy issued lands before the CTA ends
      for (int v = max(0, u - kSlots); v < u; ++v) mbar_drain(b_full + 8 * (v % kSlots), (uint32_t)(v / kSlots) & 1u);
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issuer
    // (the whole warp waits, one elected lane issues)
    constexpr uint32_t idP = idesc_bf16_f32(C, C, 0, 0);         // Q K^T: both K-major
    constexpr uint32_t idO = idesc_bf16_f32(C, DH, 0, 1);        // Q S and P V: S and V are N-major
    // K'^T V: K' in TMEM; M is 128 for DH = 64 too, lanes 64..127 of both are not used
    constexpr uint32_t idS = idesc_bf16_f32(128, DH, 0, 1);
    bool ok = true;
    auto issue_qk = [&](int c) -> bool {
      const int uq = c * kUnits, uk = uq + 1;
      if (!warp_all(full_wait(uq) && full_wait(uk))) return false;
      tc_fence_after();
      const uint64_t dq = sw128_desc(tile(uq), 16, 1024), dk = sw128_desc(tile(uk), 16, 1024);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < DH / 16; ++k) {
          const uint64_t off = (uint64_t)(((k >> 2) * L::kHalf + (k & 3) * 32) >> 4);
          umma_f16(tmem + kColP, dq + off, dk + off, idP, k > 0 ? 1u : 0u);
        }
        umma_commit(b_qk);
      }
      __syncwarp();
      return true;
    };
    if (OUT) ok = issue_qk(0);
    for (int c = 0; c < n && ok; ++c) {
      const int uk = c * kUnits + kK, uv = uk + 1;
      const uint32_t par = (uint32_t)c & 1u;
      const uint64_t dv = sw128_desc(tile(uv), L::kHalf, 1024);
      if (OUT) {
        const int uq = uk - 1;
        if (!warp_all(mbar_wait(b_s, par, s_abort) && (c == 0 || mbar_wait(b_ofree, par ^ 1u, s_abort)))) { ok = false; break; }
        tc_fence_after();
        const uint64_t dq = sw128_desc(tile(uq), 16, 1024), ds = sw128_desc(sb + L::kOffS, L::kSHalf, 1024);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < DH / 16; ++k) {
            const uint64_t off = (uint64_t)(((k >> 2) * L::kHalf + (k & 3) * 32) >> 4);
            umma_f16(tmem + kColO, dq + off, ds + (uint64_t)((k * 16 * 128) >> 4), idO, k > 0 ? 1u : 0u);
          }
          umma_commit(b_qs);
          umma_commit(b_empty + 8 * (uq % kSlots));
        }
        __syncwarp();
      }
      if (!warp_all(full_wait(uv) &&
                    (OUT || c < 2 || mbar_wait(b_sf + 8 * (c & 1), (uint32_t)((c >> 1) - 1) & 1u, s_abort)))) {
        ok = false;
        break;
      }
      const uint32_t tS = tmem + (OUT ? kColS : (uint32_t)(c & 1) * 128u);
#pragma unroll 1
      for (int part = 0; part < kParts && c < n_state; ++part) {
        const int g = c * kParts + part;
        if (!warp_all(mbar_wait(b_kp + 8 * (g & 1), (uint32_t)(g >> 1) & 1u, s_abort))) { ok = false; break; }
        tc_fence_after();
        const uint32_t ta = tmem + kColK + (uint32_t)(g & 1) * kBufCols;
        const uint64_t db = dv + (uint64_t)(part * kPart * 128 >> 4);
        if (elect_one()) {
#pragma unroll
          for (int term = 0; term < 3; ++term)
#pragma unroll
            for (int k = 0; k < kPart / 16; ++k)
              umma_f16_ts(tS, ta + term * kTermCols + k * 8, db + (uint64_t)((k * 16 * 128) >> 4), idS,
                          part + term + k > 0 ? 1u : 0u);
          umma_commit(b_kv + 8 * (g & 1));
        }
        __syncwarp();
      }
      if (!ok) break;
      if (REPAIR) {                                      // V is repaired after these products
        if (c < n_state && elect_one()) umma_commit(b_pd + 8 * (c & 1));
        __syncwarp();
      }
      // P is there and O holds the scaled Q S.  These products and the next
      // chunk's Q K^T run while the state warps bring S forward.
      if (OUT && !warp_all(mbar_wait(b_p, par, s_abort))) { ok = false; break; }
      tc_fence_after();
      if (elect_one()) {
        if (!REPAIR && c < n_state) umma_commit(b_pd + 8 * (c & 1));   // with the rest: 240 us, ahead as above: 245
        if (OUT) {
#pragma unroll
          for (int k = 0; k < C / 16; ++k)
            umma_f16_ts(tmem + kColO, tmem + kColP + k * 8, dv + (uint64_t)((k * 16 * 128) >> 4), idO, 1u);
          umma_commit(b_o);
        }
        umma_commit(b_empty + 8 * (uk % kSlots));
        umma_commit(b_empty + 8 * (uv % kSlots));
      }
      __syncwarp();
      if (OUT && c + 1 < n && !issue_qk(c + 1)) { ok = false; break; }
    }
    if (elect_one()) umma_commit(b_final);               // all MMAs done before TMEM is released
    __syncwarp();
    mbar_drain(b_final, 0);
    __syncwarp();
  } else if (warp < 4) {
    const uint32_t tl = tmem + ((uint32_t)(warp * 32) << 16);
    if (OUT) {
      // ---------------------------------------------------------- P and o
      const int i = warp * 32 + lane;                    // token row of the chunk (TMEM lane)
      // The powers each thread needs are the same for every chunk and sit in
      // registers: the products read shared memory at its full rate, and a
      // load from it waits long.  Before the diagonal a^{i - j} =
      // a^{i - 32q - 31} a^{31 - jj}; on it, 2^(log2(a) (i - j)) at P's bf16
      // precision.
      const float ai = s_pow[i + 1] * p.scale;
      // (a decay below 2^-160 a token is none of it: a^1 is zero in fp32 either
      // way, and the bound keeps the exponents' rounding below P's)
      const float l2a = ld < -110.f ? -160.f : ld * 1.4426950408889634f;
      const float top = log2f(fabsf(p.scale));           // on the diagonal: |scale| 2^(l2a (i - j)), at most |scale|
      const float base = fmaf(l2a, (float)lane, top);
      const uint32_t flip = p.scale < 0.f ? 0x80008000u : 0u;
      float row[3];
#pragma unroll
      for (int q = 0; q < 3; ++q) row[q] = s_pow[max(i - 32 * q - 31, 0)] * p.scale;
      float2 col[16];                                    // a^{31 - jj}, the same for every lane
#pragma unroll
      for (int x = 0; x < 16; ++x) col[x] = make_float2(s_pow[31 - 2 * x], s_pow[30 - 2 * x]);
      auto work_p = [&](int c) -> bool {
        if (!warp_all(mbar_wait(b_qk, (uint32_t)c & 1u, s_abort))) return false;
        tc_fence_after();
#pragma unroll
        for (int q = 0; q < 4; ++q) {                    // columns 32 q .. 32 q + 31
          uint32_t w[16];
          if (q <= warp) {                               // some column is at or before the warp's last row
            uint32_t r[32];
            tmem_ld32(tl + kColP + 32 * q, r);
            tmem_wait_ld();
            if (q < warp) {
              const float2 f2 = make_float2(row[q < 3 ? q : 0], row[q < 3 ? q : 0]);
#pragma unroll
              for (int x = 0; x < 16; ++x) {
                const float2 y = mul2(mul2(make_float2(__uint_as_float(r[2 * x]), __uint_as_float(r[2 * x + 1])), f2), col[x]);
                w[x] = pack_bf16x2(y.x, y.y);
              }
            } else {
#pragma unroll
              for (int x = 0; x < 16; ++x) {             // branch-free: a masked value is cut off by its bits
                const float e0 = fminf(fmaf(-2.f * x, l2a, base), top), e1 = fminf(fmaf(-2.f * x - 1.f, l2a, base), top);
                const float y0 = __uint_as_float(r[2 * x]) * exp2f(e0), y1 = __uint_as_float(r[2 * x + 1]) * exp2f(e1);
                w[x] = (pack_bf16x2(y0, y1) ^ flip) & (2 * x + 1 <= lane ? 0xffffffffu : 2 * x <= lane ? 0xffffu : 0u);
              }
            }
          } else {
#pragma unroll
            for (int x = 0; x < 16; ++x) w[x] = 0u;
          }
          tmem_st16(tl + kColP + 16 * q, w);             // over columns this warp has read
        }
        // O = scale a^{i+1} Q S, onto which the tensor cores add P V
        if (!warp_all(mbar_wait(b_qs, (uint32_t)c & 1u, s_abort))) return false;
        tc_fence_after();
        const float2 a2 = make_float2(ai, ai);
#pragma unroll 1
        for (int q = 0; q < DH / 32; ++q) {
          uint32_t r[32];
          tmem_ld32(tl + kColO + 32 * q, r);
          tmem_wait_ld();
#pragma unroll
          for (int x = 0; x < 32; x += 2) {
            const float2 y = mul2(a2, make_float2(__uint_as_float(r[x]), __uint_as_float(r[x + 1])));
            r[x] = __float_as_uint(y.x);
            r[x + 1] = __float_as_uint(y.y);
          }
          tmem_st32(tl + kColO + 32 * q, r);
        }
        tmem_wait_st();
        tc_fence_before();
        if (REPAIR) {
          const int uv = c * kUnits + kK + 1;
          if (!warp_all(full_wait(uv) && (c >= n_state || mbar_wait(b_pd + 8 * (c & 1), (uint32_t)(c >> 1) & 1u, s_abort))))
            return false;
          if (i < DH) {                                  // column i of V
            uint8_t* half = smem + (tile(uv) - sb) + (i / 64) * L::kHalf;
            int first = C;
            for (int j = C - 1; j >= 0; --j) {
              uint16_t* e = reinterpret_cast<uint16_t*>(half + j * 128 + ((((i & 63) / 8) ^ (j & 7)) * 16)) + (i & 7);
              if ((*e & 0x7f80u) == 0x7f80u) {
                *e = 0;
                first = j;
              }
            }
            s_first[i] = (uint8_t)first;                 // the last chunk's are read
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        mbar_arrive(b_p);
        return true;
      };
      // o through a staging tile, so that a copy writes whole rows
      auto work_o = [&](int c) {
        tc_fence_after();
#pragma unroll 2
        for (int q = 0; q < DH / 32; ++q) {
          uint32_t r[32];
          tmem_ld32(tl + kColO + 32 * q, r);
          tmem_wait_ld();
          if (REPAIR) {
#pragma unroll
            for (int x = 0; x < 32; ++x)
              if (s_first[32 * q + x] <= i) r[x] = 0x7fffffffu;
          }
          if (q + 1 == DH / 32) {
            tc_fence_before();
            mbar_arrive(b_ofree);                        // O is read
          }
          uint8_t* dst = smem + L::kOffO + (q / 2) * L::kHalf + i * 128;
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            uint32_t y[4];
#pragma unroll
            for (int x = 0; x < 4; ++x)
              y[x] = pack_bf16x2(__uint_as_float(r[8 * v + 2 * x]), __uint_as_float(r[8 * v + 2 * x + 1]));
            *reinterpret_cast<uint4*>(dst + ((((q & 1) * 4 + v) ^ (i & 7)) * 16)) = make_uint4(y[0], y[1], y[2], y[3]);
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        group_all(1, 128, true);
        if (threadIdx.x == 0) {                          // rows past the sequence are not written
#pragma unroll
          for (int hf = 0; hf < NH; ++hf)
            tma_store_4d(&tm_o, sb + L::kOffO + hf * L::kHalf, 64 * hf, h, (c0 + c) * C, b);
          asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
      };
      for (int c = 0; c < n; ++c) {
        const bool there = work_p(c) && warp_all(mbar_wait(b_o, (uint32_t)c & 1u, s_abort));
        // the copy of the chunk before has read the staging tile; the four warps
        // go on, or give up, together
        if (threadIdx.x == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        if (!group_all(1, 128, there)) break;
        work_o(c);
      }
      if (threadIdx.x == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
      if (!REPAIR && warp == 0) {                        // o of the last chunk's first token: finite?
        uint32_t over = 0u;                              // bits 15 and 31: an exponent of ones, + 1
#pragma unroll
        for (int hf = 0; hf < NH; ++hf)
          over |= (reinterpret_cast<const uint32_t*>(smem + L::kOffO + hf * L::kHalf)[lane] & 0x7f807f80u) + 0x00800080u;
        again = !group_all(2, 32 + 32 * kStateWarps, (over & 0x80008000u) == 0u || *s_abort != 0);
      }
    } else {
      // parts 0 and 2; the state warps' second half has 1 and 3
      for (int c = 0; c < n; ++c)
        if (!warp_all(full_wait(c * kUnits + kK)) || !scale_k(c, 0, 2)) break;
    }
  } else {
    // ------------------------------------------------------------ state
    constexpr int NC = DH / 2;                           // columns of S per thread
    const int tid = threadIdx.x - 128, col0 = tid / 128 * NC;
    const int r = (warp & 3) * 32 + lane;                // row of S (TMEM lane)
    const bool mine = r < DH;                            // whole warps: DH is 64 or 128
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16) + col0;
    float S[NC];
    const float* src = nullptr;                          // the state before this segment
    if (OUT) src = p.n_seg > 1 ? p.ws + ((size_t)pair * p.n_seg + seg) * DH * DH
                               : p.init != nullptr ? p.init + (size_t)pair * DH * DH : nullptr;
    if (OUT && p.n_seg > 1) asm volatile("griddepcontrol.wait;" ::: "memory");       // for combine_kernel
    [[maybe_unused]] const long long n_src = (long long)p.B * p.H * p.n_seg * DH * DH;
    const long long at = (long long)r * DH + col0;
    const bool load = mine && src != nullptr && RATP_IN(((long long)pair * p.n_seg + seg) * DH * DH + at, NC, n_src);
#pragma unroll
    for (int x = 0; x < NC; x += 4) {
      const float4 v = load ? *reinterpret_cast<const float4*>(src + at + x) : make_float4(0.f, 0.f, 0.f, 0.f);
      S[x] = v.x; S[x + 1] = v.y; S[x + 2] = v.z; S[x + 3] = v.w;
    }
    auto publish = [&]() {                               // S as bf16, [half][row][64], 128-byte swizzle
      if (mine) {
#pragma unroll
        for (int x = 0; x < NC; x += 8) {
          const int cc = col0 + x, ch = (cc & 63) / 8;
          *reinterpret_cast<uint4*>(smem + L::kOffS + (cc / 64) * L::kSHalf + r * 128 + ((ch ^ (r & 7)) * 16)) =
              make_uint4(pack_bf16x2(S[x], S[x + 1]), pack_bf16x2(S[x + 2], S[x + 3]), pack_bf16x2(S[x + 4], S[x + 5]),
                         pack_bf16x2(S[x + 6], S[x + 7]));
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(b_s);
    };
    float left = 0.f;
    // S = a^n S + chunk c's products, which are done
    auto update = [&](int c) {
      tc_fence_after();
      const Decay a = s_decay[tokens(c) == C ? 0 : 1];
      // a^n rounded so that what the roundings of the chunks so far have left out
      // is made up for: their product stays within one rounding of the power
      left = __fadd_rn(left, a.lo);
      const float m = __fadd_rn(a.hi, left);
      left = __fsub_rn(left, __fsub_rn(m, a.hi));
      const float2 power = make_float2(m, m);
      const uint32_t tc = tl + (OUT ? kColS : (uint32_t)(c & 1) * 128u);
      if (mine) {
#pragma unroll
        for (int q = 0; q < NC / 32; ++q) {
          uint32_t v[32];
          tmem_ld32(tc + 32 * q, v);
          tmem_wait_ld();
#pragma unroll
          for (int x = 0; x < 32; x += 2) {
            float* s = S + 32 * q + x;
            const float2 was = make_float2(s[0], s[1]), add = make_float2(__uint_as_float(v[x]), __uint_as_float(v[x + 1]));
            const float2 y = fma2(power, was, add);
            s[0] = y.x;
            s[1] = y.y;
          }
        }
      }
      tc_fence_before();
    };
    auto products = [&](int c) { return warp_all(mbar_wait(b_pd + 8 * (c & 1), (uint32_t)(c >> 1) & 1u, s_abort)); };
    bool ok = true;
    if (OUT) {
      publish();
      for (int c = 0; c < n_state; ++c) {
        if (!warp_all(full_wait(c * kUnits + kK)) || !scale_k(c, tid / 128, 2) || !products(c)) {
          ok = false;
          break;
        }
        update(c);
        if (c + 1 < n) publish();
      }
    } else {
      // the second half's scaling runs one chunk ahead of its update
      for (int c = 0; c <= n; ++c) {
        if ((tid >= 128 && c < n && (!warp_all(full_wait(c * kUnits + kK)) || !scale_k(c, 1, 2))) ||
            (c > 0 && !products(c - 1))) {
          ok = false;
          break;
        }
        if (c > 0) {
          update(c - 1);
          mbar_arrive(b_sf + 8 * ((c - 1) & 1));
        }
      }
    }
    // a state that will be computed again is not written: it may lie where the
    // initial one is read from
    if (OUT && !REPAIR) again = !group_all(2, 32 + 32 * kStateWarps, true);
    float* dst = OUT ? (want_end ? p.fin + (size_t)pair * DH * DH : nullptr)
                     : p.ws + ((size_t)pair * p.n_seg + seg) * DH * DH;
    if (ok && !again && mine && dst != nullptr) {
#pragma unroll
      for (int x = 0; x < NC; x += 4)
        *reinterpret_cast<float4*>(dst + at + x) = make_float4(S[x], S[x + 1], S[x + 2], S[x + 3]);
    }
  }

  tc_fence_before();
  const bool any = __syncthreads_or(again);
  tc_fence_after();
  return any;
}

template <int DH>
__device__ __noinline__ void repair_pass(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                         const CUtensorMap& tm_o, const Params& p, uint8_t* smem, uint32_t tmem) {
  chunk_pass<DH, true, true>(tm_q, tm_k, tm_v, tm_o, p, smem, tmem);
}

template <int DH, bool OUT>
__global__ void __launch_bounds__(kThreads, 1)
chunk_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
             const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o,
             const __grid_constant__ Params p) {
  using namespace sm100;
  using L = Layout<DH>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* s_pow = reinterpret_cast<float*>(smem + L::kOffPow);
  Decay* s_decay = reinterpret_cast<Decay*>(smem + L::kOffDecay);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + L::kOffCtl);
  if (!OUT) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = threadIdx.x >> 5;
  const int per = OUT ? p.n_seg : p.n_seg - 1, pair = blockIdx.x / per;
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(s_tmem), kTmemCols);
    tmem_relinquish();
  }
  const float ld = p.log_decay[pair % p.H];
  if (threadIdx.x == 0) {
    *reinterpret_cast<volatile int*>(smem + L::kOffCtl + 4) = 0;
    if (!(ld <= 0.f)) raise_error(RATP_ERR_ARG);
  }
  if (threadIdx.x <= C) s_pow[threadIdx.x] = decay_power(ld, (double)threadIdx.x);
  else if (threadIdx.x <= C + 2)
    s_decay[threadIdx.x - C - 1] = decay_pair(ld, threadIdx.x == C + 1 ? (double)C : (double)(p.T - (p.n_chunks - 1) * C));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  const bool again = chunk_pass<DH, OUT, false>(tm_q, tm_k, tm_v, tm_o, p, smem, tmem);
  if constexpr (OUT) {
    if (again) repair_pass<DH>(tm_q, tm_k, tm_v, tm_o, p, smem, tmem);
  }
  if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

// Segment states -> the state before each segment, in place: element e of
// (b, h) walks its segments.  grid (ceil(DH * DH / 4 / 256), B * H).
__global__ void __launch_bounds__(256)
combine_kernel(float* __restrict__ ws, const float* __restrict__ init, const float* __restrict__ log_decay, int H,
               int h0, int n_seg, int quads, int seg_tokens, [[maybe_unused]] long long n_ws) {
  const int e = blockIdx.x * 256 + threadIdx.x, pair = blockIdx.y;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (e >= quads) return;
  const Decay a = decay_pair(log_decay[(h0 + pair) % H], (double)seg_tokens);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float4* w = reinterpret_cast<float4*>(ws) + (long long)pair * n_seg * quads + e;
  if (!RATP_IN(((long long)pair * n_seg * quads + e) * 4, ((long long)(n_seg - 1) * quads + 1) * 4, n_ws)) return;
  float4 run = init != nullptr ? reinterpret_cast<const float4*>(init)[(long long)pair * quads + e]
                               : make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int kBatch = 8;                              // segments whose loads are in flight at once
  for (int s0 = 0; s0 < n_seg; s0 += kBatch) {
    float4 own[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      own[i] = s0 + i + 1 < n_seg ? w[(long long)(s0 + i) * quads] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (s0 + i >= n_seg) break;
      w[(long long)(s0 + i) * quads] = run;
      run.x = a.step(run.x, own[i].x);
      run.y = a.step(run.y, own[i].y);
      run.z = a.step(run.z, own[i].z);
      run.w = a.step(run.w, own[i].w);
    }
  }
}

// ---- token by token -------------------------------------------------------------
// A CTA holds 64 columns (dv) of one (b, h)'s state in registers: thread
// (row group of 16 lanes, 4 columns) has rows dk = g, g + 16, ...  q . S is
// summed over the rows by shuffles and shared memory.
struct RecurrentParams {
  const __nv_bfloat16 *q, *k, *v;      // [B][T][H][DH]
  __nv_bfloat16* o;
  const float* log_decay;
  const float* init;                   // may be fin (in place), or NULL
  float* fin;                          // or NULL
  int B, T, H;
  float scale;
};

template <int DH>
__global__ void __launch_bounds__(256)
recurrent_kernel(const RecurrentParams p) {
  constexpr int kRows = DH / 16;                         // rows per thread
  __shared__ float s_q[DH], s_k[DH];
  __shared__ float s_o[8][64];
  const int pair = blockIdx.x / (DH / 64), c0 = (blockIdx.x % (DH / 64)) * 64;
  const int b = pair / p.H, h = pair - b * p.H;
  const int g = threadIdx.x / 16, col = c0 + (threadIdx.x % 16) * 4;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long s0 = (long long)pair * DH * DH + col;
  [[maybe_unused]] const long long n_s = (long long)p.B * p.H * DH * DH;
  [[maybe_unused]] const long long n_tok = (long long)p.B * p.T * p.H * DH;
  float4 S[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const long long at = s0 + (long long)(g + 16 * i) * DH;
    S[i] = p.init != nullptr && RATP_IN(at, 4, n_s) ? __ldcs(reinterpret_cast<const float4*>(p.init + at))
                                                    : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const float ld = p.log_decay[h];
  if (!(ld <= 0.f) && threadIdx.x == 0) raise_error(RATP_ERR_ARG);
  const Decay a = decay_pair(ld, 1.0);
  for (int t = 0; t < p.T; ++t) {
    const long long row = (((long long)b * p.T + t) * p.H + h) * DH;
    const bool in = RATP_IN(row, DH, n_tok);
    if (t > 0) __syncthreads();                          // s_q, s_k, s_o of the token before are read
    if (threadIdx.x < DH) s_q[threadIdx.x] = in ? __bfloat162float(p.q[row + threadIdx.x]) * p.scale : 0.f;
    else if (threadIdx.x < 2 * DH) s_k[threadIdx.x - DH] = in ? __bfloat162float(p.k[row + threadIdx.x - DH]) : 0.f;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (in) {
      const uint2 x = *reinterpret_cast<const uint2*>(p.v + row + col);
      v[0] = __uint_as_float(x.x << 16); v[1] = __uint_as_float(x.x & 0xffff0000u);
      v[2] = __uint_as_float(x.y << 16); v[3] = __uint_as_float(x.y & 0xffff0000u);
    }
    __syncthreads();
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const float k = s_k[g + 16 * i], q = s_q[g + 16 * i];
      S[i].x = a.step(S[i].x, k * v[0]);
      S[i].y = a.step(S[i].y, k * v[1]);
      S[i].z = a.step(S[i].z, k * v[2]);
      S[i].w = a.step(S[i].w, k * v[3]);
      o.x = fmaf(q, S[i].x, o.x);
      o.y = fmaf(q, S[i].y, o.y);
      o.z = fmaf(q, S[i].z, o.z);
      o.w = fmaf(q, S[i].w, o.w);
    }
    if (t + 1 == p.T && p.fin != nullptr) {
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const long long at = s0 + (long long)(g + 16 * i) * DH;
        if (RATP_IN(at, 4, n_s)) __stcs(reinterpret_cast<float4*>(p.fin + at), S[i]);
      }
    }
    o.x += __shfl_xor_sync(0xffffffffu, o.x, 16);
    o.y += __shfl_xor_sync(0xffffffffu, o.y, 16);
    o.z += __shfl_xor_sync(0xffffffffu, o.z, 16);
    o.w += __shfl_xor_sync(0xffffffffu, o.w, 16);
    if (lane < 16) {
      s_o[warp][lane * 4] = o.x;
      s_o[warp][lane * 4 + 1] = o.y;
      s_o[warp][lane * 4 + 2] = o.z;
      s_o[warp][lane * 4 + 3] = o.w;
    }
    __syncthreads();
    if (threadIdx.x < 32 && in) {
      float y[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        y[j] = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) y[j] += s_o[w][2 * lane + j];
      }
      *reinterpret_cast<uint32_t*>(p.o + row + c0 + 2 * lane) = pack_bf16x2(y[0], y[1]);
    }
  }
}

}  // namespace linear_attn
}  // namespace ratp
