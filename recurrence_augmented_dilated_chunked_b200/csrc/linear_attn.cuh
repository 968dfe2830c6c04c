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
//   all its time.
// * chunk_kernel takes 128 tokens at a time on the tensor cores.  With S the
//   state before the chunk, n the tokens in it, i, j = 0 .. n-1:
//     o_i  = scale (a^{i+1} q_i S + sum_{j <= i} a^{i-j} (q_i . k_j) v_j)
//     S'   = a^n S + sum_j a^{n-1-j} k_j v_j^T
//   that is, with P = mask(Q K^T) * a^{i-j}: two products read against the
//   chunk's values and state, and one that advances the state.
//   No power of a is ever inverted, so any decay in (0, 1] is as exact as any
//   other.  P and the state enter their products rounded to bf16 (as the
//   attention's P does: the output is bf16 itself).  The state's own update
//   keeps 16 bits of a^{n-1-j} k_j as two bf16 terms (hi + lo, two products),
//   the products accumulate one chunk only, and the running state is fp32 in
//   registers, so the state that is handed on is exact to fp32's order.
//
// A sequence is a chain over its chunks, so few (b, h) leave SMs idle: then
// the chunks are cut into segments.  chunk_kernel<DH, false> computes every
// segment's own state (from zero), combine_kernel turns those into the state
// before each segment, and chunk_kernel<DH, true> runs all segments at once.
//
// Roles of chunk_kernel (320 threads, one CTA per SM):
//   warps 0-3  P: read Q K^T from TMEM, mask, decay, write bf16 P to TMEM over
//              it; then o = scale (a^{i+1} O1 + O2) out of TMEM to memory;
//   warps 4-7  state: scale K in place to its hi part, lo part beside it; then
//              S = a^n S + (TMEM) in registers, and S as bf16 in shared memory;
//   warp 8     TMA producer: K, Q, V tiles through a ring of kSlots tiles;
//   warp 9     TMEM and the MMA issuer.  Per chunk: P = Q K^T (M 128 tokens, N
//              128 tokens), O1 = Q S, SL = K'^T V (M = Dh, hi then lo), O2 = P V.
//   Without an output (<DH, false>) only SL is computed, and warps 0-3 share
//   the scaling of K.
// Bound: 4 tiles of memory traffic per chunk and (b, h) against five products.
#pragma once
#include "sm100.cuh"

namespace ratp {
namespace linear_attn {

constexpr int C = 128;                 // tokens per chunk
constexpr int kThreads = 320;
constexpr int kProducerWarp = 8;
constexpr int kMmaWarp = 9;
constexpr int kSlots = 5;
constexpr int kRecurrentTokens = 16;

// a^n for n >= 0 tokens.  log_decay is clamped to a finite value, below which
// every power but the 0th is zero in fp32.
__device__ __forceinline__ float decay_power(float log_decay, double n) {
  return n == 0.0 ? 1.f : (float)exp(fmax((double)log_decay, -1.0e4) * n);
}

template <int DH>
struct Layout {
  static constexpr uint32_t kHalf = C * 128;             // 128 rows x 64 bf16
  static constexpr uint32_t kTile = (DH / 64) * kHalf;
  static constexpr uint32_t kOffLo = kSlots * kTile;     // K's lo part
  static constexpr uint32_t kOffS = kOffLo + kTile;      // S, bf16 [DH / 64][DH rows][64]
  static constexpr uint32_t kSHalf = DH * 128;
  static constexpr uint32_t kOffPow = kOffS + (DH / 64) * kSHalf;    // a^0 .. a^128
  static constexpr uint32_t kOffBar = kOffPow + (C + 1) * 4 + 4;
  static constexpr int kBars = 2 * kSlots + 8;
  static constexpr uint32_t kOffCtl = kOffBar + kBars * 8;           // TMEM address, abort flag
  // one CTA per SM whatever DH, since each takes all of TMEM
  static constexpr uint32_t kBytes = (kOffCtl + 8 + 1024) > 120 * 1024 ? (kOffCtl + 8 + 1024) : 120 * 1024;
};
static_assert(Layout<128>::kBytes <= 232448, "shared memory of one CTA");

constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColP = 0;          // 128 columns: Q K^T, then P as bf16 pairs in the first 64

struct Params {
  __nv_bfloat16* o;
  const float* log_decay;              // [H]
  const float* init;                   // [B][H][DH][DH] or NULL: the state before the sequence
  float* fin;                          // [B][H][DH][DH] or NULL: the state after it
  float* ws;                           // [B * H][n_seg][DH][DH]: segment states
  int B, T, H;
  int n_chunks, seg_chunks, n_seg;
  float scale;
  int o_align32;
};

// Two floats as bf16 pairs: hi the rounded values, lo what they leave.
__device__ __forceinline__ void split2(float2 x, float2 w, uint32_t* hi, uint32_t* lo) {
  const float2 y = mul2(x, w);
  *hi = pack_bf16x2(y.x, y.y);
  const float2 h = make_float2(__uint_as_float(*hi << 16), __uint_as_float(*hi & 0xffff0000u));
  const float2 r = fma2(x, w, make_float2(-h.x, -h.y));
  *lo = pack_bf16x2(r.x, r.y);
}

template <int DH, bool OUT>
__global__ void __launch_bounds__(kThreads, 1)
chunk_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
             const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ Params p) {
  using namespace sm100;
  using L = Layout<DH>;
  constexpr int NH = DH / 64;                            // 64-channel halves
  constexpr int kUnits = OUT ? 3 : 2;                    // tiles per chunk: K, (Q,) V
  constexpr uint32_t kColO1 = 128, kColO2 = kColO1 + DH, kColS = kColO2 + DH;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  const uint32_t bar0 = sb + L::kOffBar;
  const uint32_t b_full = bar0, b_empty = bar0 + 8 * kSlots;
  const uint32_t b_qk = bar0 + 8 * (2 * kSlots), b_p = b_qk + 8, b_o = b_qk + 16, b_ofree = b_qk + 24;
  const uint32_t b_kp = b_qk + 32, b_kv = b_qk + 40, b_s = b_qk + 48, b_final = b_qk + 56;
  float* s_pow = reinterpret_cast<float*>(smem + L::kOffPow);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + L::kOffCtl);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + L::kOffCtl + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

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
    *s_abort = 0;
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(b_full + 8 * i, 1);
      mbar_init(b_empty + 8 * i, 1);
    }
    mbar_init(b_qk, 1);
    mbar_init(b_p, 128);
    mbar_init(b_o, 1);
    mbar_init(b_ofree, 128);
    mbar_init(b_kp, OUT ? 128 : 256);
    mbar_init(b_kv, 1);
    mbar_init(b_s, 128);
    mbar_init(b_final, 1);
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(s_tmem), kTmemCols);
    tmem_relinquish();
  }
  const float ld = p.log_decay[h];
  if (threadIdx.x <= C) s_pow[threadIdx.x] = decay_power(ld, (double)threadIdx.x);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;

  // tile u of this CTA (chunk u / kUnits; K, (Q,) V in turn) lies in slot u % kSlots
  auto full_wait = [&](int u) { return mbar_wait(b_full + 8 * (u % kSlots), (uint32_t)(u / kSlots) & 1u, s_abort); };
  auto tile = [&](int u) { return sb + (uint32_t)(u % kSlots) * L::kTile; };

  // a^{n-1-j} k_j of chunk c, hi in place and lo beside it, by threads
  // tid + part * 128 of parts * 128; zero rows past the sequence stay zero
  auto scale_k = [&](int c, int tid, int part, int parts) {
    const int m = tokens(c);
    uint8_t* t = smem + (uint32_t)((c * kUnits) % kSlots) * L::kTile;
    uint8_t* lo = smem + L::kOffLo;
#pragma unroll 4
    for (int i = part; i < NH * 8; i += parts) {
      const int row = (i & 7) * 16 + tid / 8;            // 16 bytes of row `row`, half i / 8 (swizzled within it)
      const uint32_t off = (uint32_t)(i * 128 + tid) * 16;
      const float w = s_pow[max(m - 1 - row, 0)];
      const float2 w2 = make_float2(w, w);
      float2 f[4];
      Elem<__nv_bfloat16>::unpack2(*reinterpret_cast<const uint4*>(t + off), f);
      uint4 hv, lv;
      split2(f[0], w2, &hv.x, &lv.x);
      split2(f[1], w2, &hv.y, &lv.y);
      split2(f[2], w2, &hv.z, &lv.z);
      split2(f[3], w2, &hv.w, &lv.w);
      *reinterpret_cast<uint4*>(t + off) = hv;
      *reinterpret_cast<uint4*>(lo + off) = lv;
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
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
          const CUtensorMap* m = i == 0 ? &tm_k : i == kUnits - 1 ? &tm_v : &tm_q;
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
    if (lane == 0) {
      constexpr uint32_t idP = idesc_bf16_f32(C, C, 0, 0);       // Q K^T: both K-major
      constexpr uint32_t idO1 = idesc_bf16_f32(C, DH, 0, 1);     // Q S: S is [dk][dv], N-major
      constexpr uint32_t idO2 = idesc_bf16_f32(C, DH, 0, 1);     // P V: P in TMEM
      constexpr uint32_t idS = idesc_bf16_f32(128, DH, 1, 1);    // K'^T V: K' is [token][dk], M-major
      // M is 128 for DH = 64 too: both halves of M read the same 64 channels,
      // and lanes 64..127 of the result are not used
      constexpr uint32_t kMHalf = DH == 128 ? L::kHalf : 0;
      bool ok = true;
      for (int c = 0; c < n && ok; ++c) {
        const int uk = c * kUnits, uv = uk + kUnits - 1;
        const uint32_t par = (uint32_t)c & 1u;
        if (OUT) {
          const int uq = uk + 1;
          if (!full_wait(uk) || !full_wait(uq)) { ok = false; break; }
          tc_fence_after();
          const uint64_t dq = sw128_desc(tile(uq), 16, 1024), dk = sw128_desc(tile(uk), 16, 1024);
#pragma unroll
          for (int k = 0; k < DH / 16; ++k) {
            const uint64_t off = (uint64_t)(((k >> 2) * L::kHalf + (k & 3) * 32) >> 4);
            umma_f16(tmem + kColP, dq + off, dk + off, idP, k > 0 ? 1u : 0u);
          }
          umma_commit(b_qk);
          if (!mbar_wait(b_s, par, s_abort) || (c > 0 && !mbar_wait(b_ofree, par ^ 1u, s_abort))) { ok = false; break; }
          tc_fence_after();
          const uint64_t ds = sw128_desc(sb + L::kOffS, L::kSHalf, 1024);
#pragma unroll
          for (int k = 0; k < DH / 16; ++k) {
            const uint64_t off = (uint64_t)(((k >> 2) * L::kHalf + (k & 3) * 32) >> 4);
            umma_f16(tmem + kColO1, dq + off, ds + (uint64_t)((k * 16 * 128) >> 4), idO1, k > 0 ? 1u : 0u);
          }
          umma_commit(b_empty + 8 * (uq % kSlots));
        }
        const uint64_t dv = sw128_desc(tile(uv), L::kHalf, 1024);
        if (c < n_state) {
          if (!mbar_wait(b_kp, par, s_abort) || !full_wait(uv)) { ok = false; break; }
          tc_fence_after();
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            const uint64_t da = sw128_desc(part == 0 ? tile(uk) : sb + L::kOffLo, kMHalf, 1024);
#pragma unroll
            for (int k = 0; k < C / 16; ++k)
              umma_f16(tmem + kColS, da + (uint64_t)((k * 16 * 128) >> 4), dv + (uint64_t)((k * 16 * 128) >> 4), idS,
                       part + k > 0 ? 1u : 0u);
          }
          umma_commit(b_kv);
        }
        umma_commit(b_empty + 8 * (uk % kSlots));
        if (OUT) {
          if (!mbar_wait(b_p, par, s_abort) || !full_wait(uv)) { ok = false; break; }
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < C / 16; ++k)
            umma_f16_ts(tmem + kColO2, tmem + kColP + k * 8, dv + (uint64_t)((k * 16 * 128) >> 4), idO2, k > 0 ? 1u : 0u);
          umma_commit(b_o);
        }
        umma_commit(b_empty + 8 * (uv % kSlots));
      }
      umma_commit(b_final);                              // all MMAs done before TMEM is released
      mbar_drain(b_final, 0);
    }
    __syncwarp();
  } else if (warp < 4) {
    const uint32_t tl = tmem + ((uint32_t)(warp * 32) << 16);
    if (OUT) {
      // ---------------------------------------------------------- P and o
      const int i = warp * 32 + lane;                    // token row of the chunk (TMEM lane)
      const float ai = s_pow[i + 1] * p.scale;
      float2 col[16];                                    // a^{31 - jj}, the same for every lane
#pragma unroll
      for (int x = 0; x < 16; ++x) col[x] = make_float2(s_pow[31 - 2 * x], s_pow[30 - 2 * x]);
      for (int c = 0; c < n; ++c) {
        const uint32_t par = (uint32_t)c & 1u;
        if (!warp_all(mbar_wait(b_qk, par, s_abort))) break;
        tc_fence_after();
#pragma unroll
        for (int q = 0; q < 4; ++q) {                    // columns 32 q .. 32 q + 31
          uint32_t w[16];
          if (q <= warp) {                               // some column is at or before the warp's last row
            uint32_t r[32];
            tmem_ld32(tl + kColP + 32 * q, r);
            tmem_wait_ld();
            if (q < warp) {
              const float f = s_pow[i - 32 * q - 31];    // a^{i - j} = a^{i - 32q - 31} a^{31 - jj}
              const float2 f2 = make_float2(f, f);
#pragma unroll
              for (int x = 0; x < 16; ++x) {
                const float2 y = mul2(make_float2(__uint_as_float(r[2 * x]), __uint_as_float(r[2 * x + 1])), mul2(f2, col[x]));
                w[x] = pack_bf16x2(y.x, y.y);
              }
            } else {
#pragma unroll
              for (int x = 0; x < 16; ++x) {
                const int d0 = lane - 2 * x, d1 = d0 - 1;
                const float y0 = d0 >= 0 ? __uint_as_float(r[2 * x]) * s_pow[max(d0, 0)] : 0.f;
                const float y1 = d1 >= 0 ? __uint_as_float(r[2 * x + 1]) * s_pow[max(d1, 0)] : 0.f;
                w[x] = pack_bf16x2(y0, y1);
              }
            }
          } else {
#pragma unroll
            for (int x = 0; x < 16; ++x) w[x] = 0u;
          }
          tmem_st16(tl + kColP + 16 * q, w);             // over columns this warp has read
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(b_p);
        if (!warp_all(mbar_wait(b_o, par, s_abort))) break;
        tc_fence_after();
        const int t = (c0 + c) * C + i;
        __nv_bfloat16* orow = p.o + (((size_t)b * p.T + t) * p.H + h) * DH;
        const bool there = t < p.T && RATP_IN((((long long)b * p.T + t) * p.H + h) * DH, DH, (long long)p.B * p.T * p.H * DH);
#pragma unroll 1
        for (int q = 0; q < DH / 32; ++q) {
          uint32_t r1[32], r2[32];
          tmem_ld32(tl + kColO1 + 32 * q, r1);
          tmem_ld32(tl + kColO2 + 32 * q, r2);
          tmem_wait_ld();
          if (there) {
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              uint32_t y[8];
#pragma unroll
              for (int x = 0; x < 8; ++x) {
                const int e = 16 * v + 2 * x;
                y[x] = pack_bf16x2(fmaf(ai, __uint_as_float(r1[e]), p.scale * __uint_as_float(r2[e])),
                                   fmaf(ai, __uint_as_float(r1[e + 1]), p.scale * __uint_as_float(r2[e + 1])));
              }
              __nv_bfloat16* dst = orow + 32 * q + 16 * v;
              if (p.o_align32) {
                asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                             :: "l"(dst), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3]), "r"(y[4]), "r"(y[5]), "r"(y[6]), "r"(y[7])
                             : "memory");
              } else {
                *reinterpret_cast<uint4*>(dst) = make_uint4(y[0], y[1], y[2], y[3]);
                *reinterpret_cast<uint4*>(dst + 8) = make_uint4(y[4], y[5], y[6], y[7]);
              }
            }
          }
        }
        tc_fence_before();
        mbar_arrive(b_ofree);
      }
    } else {
      for (int c = 0; c < n; ++c) {
        // K's tile is there, and lo was read by the chunk before
        if (!warp_all(full_wait(c * kUnits) && (c == 0 || mbar_wait(b_kv, (uint32_t)(c - 1) & 1u, s_abort)))) break;
        scale_k(c, threadIdx.x, 0, 2);
        mbar_arrive(b_kp);
      }
    }
  } else {
    // ------------------------------------------------------------ state
    const int tid = threadIdx.x - 128, sw = warp - 4;
    const int r = sw * 32 + lane;                        // row of S (TMEM lane)
    const bool mine = r < DH;                            // whole warps: DH is 64 or 128
    const uint32_t tl = tmem + ((uint32_t)(sw * 32) << 16) + kColS;
    float S[DH];
    const float* src = nullptr;                          // the state before this segment
    if (OUT) src = p.n_seg > 1 ? p.ws + ((size_t)pair * p.n_seg + seg) * DH * DH
                               : p.init != nullptr ? p.init + (size_t)pair * DH * DH : nullptr;
    [[maybe_unused]] const long long n_src = (long long)p.B * p.H * p.n_seg * DH * DH;
    const bool load = mine && src != nullptr && RATP_IN(((long long)pair * p.n_seg + (p.n_seg > 1 ? seg : 0)) * DH * DH + r * DH, DH, n_src);
#pragma unroll
    for (int x = 0; x < DH; x += 4) {
      const float4 v = load ? *reinterpret_cast<const float4*>(src + r * DH + x) : make_float4(0.f, 0.f, 0.f, 0.f);
      S[x] = v.x; S[x + 1] = v.y; S[x + 2] = v.z; S[x + 3] = v.w;
    }
    auto publish = [&]() {                               // S as bf16, [half][row][64], 128-byte swizzle
      if (mine) {
#pragma unroll
        for (int x = 0; x < DH; x += 8) {
          const int ch = (x & 63) / 8;
          *reinterpret_cast<uint4*>(smem + L::kOffS + (x / 64) * L::kSHalf + r * 128 + ((ch ^ (r & 7)) * 16)) =
              make_uint4(pack_bf16x2(S[x], S[x + 1]), pack_bf16x2(S[x + 2], S[x + 3]), pack_bf16x2(S[x + 4], S[x + 5]),
                         pack_bf16x2(S[x + 6], S[x + 7]));
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(b_s);
    };
    if (OUT) publish();
    bool ok = true;
    for (int c = 0; c < n_state; ++c) {
      const uint32_t par = (uint32_t)c & 1u;
      // K's tile is there; Q K^T has read it; lo was read before the last update
      if (!warp_all(full_wait(c * kUnits) && (!OUT || mbar_wait(b_qk, par, s_abort)))) { ok = false; break; }
      scale_k(c, tid, OUT ? 0 : 1, OUT ? 1 : 2);
      tc_fence_before();
      mbar_arrive(b_kp);
      if (!warp_all(mbar_wait(b_kv, par, s_abort))) { ok = false; break; }
      tc_fence_after();
      const float a = s_pow[tokens(c)];
      if (mine) {
#pragma unroll
        for (int q = 0; q < DH / 32; ++q) {
          uint32_t v[32];
          tmem_ld32(tl + 32 * q, v);
          tmem_wait_ld();
#pragma unroll
          for (int x = 0; x < 32; ++x) S[32 * q + x] = fmaf(a, S[32 * q + x], __uint_as_float(v[x]));
        }
      }
      if (OUT && c + 1 < n) publish();
    }
    float* dst = OUT ? (want_end ? p.fin + (size_t)pair * DH * DH : nullptr)
                     : p.ws + ((size_t)pair * p.n_seg + seg) * DH * DH;
    if (ok && mine && dst != nullptr) {
#pragma unroll
      for (int x = 0; x < DH; x += 4)
        *reinterpret_cast<float4*>(dst + r * DH + x) = make_float4(S[x], S[x + 1], S[x + 2], S[x + 3]);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Segment states -> the state before each segment, in place: element e of
// (b, h) walks its segments.  grid (ceil(DH * DH / 4 / 256), B * H).
__global__ void __launch_bounds__(256)
combine_kernel(float* __restrict__ ws, const float* __restrict__ init, const float* __restrict__ log_decay, int H,
               int h0, int n_seg, int quads, int seg_tokens, [[maybe_unused]] long long n_ws) {
  const int e = blockIdx.x * 256 + threadIdx.x, pair = blockIdx.y;
  if (e >= quads) return;
  const float a = decay_power(log_decay[(h0 + pair) % H], (double)seg_tokens);
  float4* w = reinterpret_cast<float4*>(ws) + (long long)pair * n_seg * quads + e;
  if (!RATP_IN(((long long)pair * n_seg * quads + e) * 4, ((long long)(n_seg - 1) * quads + 1) * 4, n_ws)) return;
  float4 run = init != nullptr ? reinterpret_cast<const float4*>(init)[(long long)pair * quads + e]
                               : make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s = 0; s < n_seg; ++s) {
    const float4 own = s + 1 < n_seg ? w[(long long)s * quads] : make_float4(0.f, 0.f, 0.f, 0.f);
    w[(long long)s * quads] = run;
    run.x = fmaf(a, run.x, own.x);
    run.y = fmaf(a, run.y, own.y);
    run.z = fmaf(a, run.z, own.z);
    run.w = fmaf(a, run.w, own.w);
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
  const float a = decay_power(p.log_decay[h], 1.0);
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
      S[i].x = fmaf(a, S[i].x, k * v[0]);
      S[i].y = fmaf(a, S[i].y, k * v[1]);
      S[i].z = fmaf(a, S[i].z, k * v[2]);
      S[i].w = fmaf(a, S[i].w, k * v[3]);
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
