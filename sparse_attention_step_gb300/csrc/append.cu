// The new tokens of a step, from the projections to the cache: RMS norm of
// every query and key head, rotation by position, queries written out, keys
// and values written to the cache rows their slots name -- in one pass.
//
//   y = x * rsqrt(mean(x^2) + eps) * (w_offset + w)
//   (a, b) -> (a cos t - b sin t, b cos t + a sin t),  t = position * inv_freq[i]
// for the pairs (a, b) of the first rotary_dim dims: dims (i, i + rotary_dim/2)
// or, interleaved, (2i, 2i + 1). e4m3 caches store code = e4m3(y / s) and
// s = max(max|y|, 2^-100) / 448 for each row of 128.
//
// Bound by HBM: every row (a head of a token) is read once and written once.
// A half-warp takes a row, 8 dims a lane, so the norm is 8 products and four
// shuffles, and a row's partner dims sit in one other lane. With
//   out_j = r * (x_j A_j + xp_j B_j),  r = rsqrt(mean + eps),
//   A_j = w_j cos t,  B_j = -+ w_p sin t   (p: the partner of j)
// A and B depend on the token and on whether the row is a query or a key, not
// on the head, so they stay in registers from head to head. A CTA takes two tokens
// (one a half-warp) and a run of the heads, [queries | keys | values] end to end, its
// four warps taking turns; each thread computes one angle of the two tokens. A
// warp's rows come through a ring in shared memory (cp.async, Raw8::kAhead rows of both
// tokens on their way), which leaves the registers to eight CTAs an SM. All of
// it is fp32, two elements an instruction (f32x2); the output type's rounding is the
// only one.
// 8192 tokens x (64 + 16) heads, bf16, pages in random order: 58.0 us, 5.79 TB/s (a
// plain copy of the same bytes: 50.5). Steps: angles a lane, rows in registers,
// two tokens' heads in unequal runs 74 us; CTAs of equal runs, angles shared 64;
// the ring 57.6, angles exact for any inv_freq 58.0. It stays short of the copy by its instructions (half of the issue
// slots) and its stores of single rows.
//
// Angles: fp32 products lose a far token's angle (at position 2^20 an fp32
// angle of 1 rad per token is off by 0.06 rad). inv_freq / 2 pi is taken once
// a thread as a 64-bit fixed-point fraction of a turn (24-bit mantissa times
// the bits of 1 / 2 pi that matter, in integers), position times it wraps modulo one turn
// by itself, and the 32 leading bits go to sincospif: off by at most 2^-24 half
// turns (the rounding of that fraction to fp32) at any position and any finite inv_freq.
#include <cuda_fp8.h>

#include <type_traits>

#include "kernels.cuh"

namespace msa {

namespace {

constexpr int kAppendWarps = 4;
constexpr int kAppendThreads = 32 * kAppendWarps;
constexpr float kE4m3Max = 448.f;
constexpr float kMinRowMax = 7.888609052210118e-31f;  // 2^-100: keeps 448 / max finite and zero rows zero

// Two fp32 values in a register pair, and their products and sums.
using f32x2 = uint64_t;
__device__ inline f32x2 pack2(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ inline void unpack2(f32x2 v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ inline f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ inline f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Eight dims of a row as stored: kWords 32-bit words.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  static constexpr int kWords = 4, kAhead = 8;
  uint32_t w[4];
  __device__ void load(const __nv_bfloat16* p) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  }
  __device__ void unpack(f32x2 (&x)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = pack2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
  }
  __device__ static void store(__nv_bfloat16* p, const f32x2 (&x)[4]) {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float lo, hi;
      unpack2(x[i], lo, hi);
      o[i] = pack_bf16(lo, hi);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(o[0], o[1], o[2], o[3]);
  }
};
template <>
struct Raw8<float> {
  static constexpr int kWords = 8, kAhead = 4;
  uint32_t w[8];
  __device__ void load(const float* p) {
    const uint4 a = reinterpret_cast<const uint4*>(p)[0], b = reinterpret_cast<const uint4*>(p)[1];
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
  }
  __device__ void unpack(f32x2 (&x)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = pack2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
  }
  __device__ static void store(float* p, const f32x2 (&x)[4]) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) unpack2(x[i], f[2 * i], f[2 * i + 1]);
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
};

// 1 / 2 pi to 256 bits, leading word first (selected, not loaded: a table in memory
// costs a call of one step 0.4 us).
__device__ inline uint64_t inv_two_pi_word(int i) {
  return i <= 0   ? 0x28be60db9391054aull
         : i == 1 ? 0x7f09d5f47d4d3770ull
         : i == 2 ? 0x36d8a5664f10e410ull
                  : 0x7f9458eaf7aef158ull;
}
// 64 bits of 1 / 2 pi from bit `at` after the point on (zeros before the first), -64 <= at < 192.
__device__ inline uint64_t inv_two_pi(int at) {
  const int sh = at & 63;
  const uint64_t hi = at < 0 ? 0 : inv_two_pi_word(at >> 6), lo = inv_two_pi_word((at >> 6) + 1);
  return sh == 0 ? hi : (hi << sh) | (lo >> (64 - sh));
}

// inv_freq / 2 pi in units of 2^-64 turn, modulo one turn: x = m 2^e with a 24-bit m,
// and whole turns of m times the bits of 2^e / 2 pi before the point drop out, so that
// the 128 bits after it are enough for any finite x (Payne and Hanek's reduction).
// Off by less than one unit: times a position, by at most 2^-33 turn.
__device__ inline uint64_t turns_per_token(float x) {
  const uint32_t u = __float_as_uint(x);
  const int be = (u >> 23) & 0xff;
  const uint32_t m = be == 0 ? (u & 0x7fffffu) : ((u & 0x7fffffu) | 0x800000u);
  const int e = (be == 0 ? 1 : be) - 150;  // -149 .. 104 (not a number: 105, its angle is not used)
  const uint64_t whole = e < -64 ? 0 : m * inv_two_pi(e);
  const uint64_t f = whole + (e < -128 ? 0 : __umul64hi(m, inv_two_pi(e + 64)));
  return (u >> 31) ? 0 - f : f;
}

template <typename T>
__device__ inline void unpack8(const Raw8<T>& r, float (&x)[8]) {
  f32x2 v[4];
  r.unpack(v);
#pragma unroll
  for (int j = 0; j < 4; ++j) unpack2(v[j], x[2 * j], x[2 * j + 1]);
}

// What a lane keeps from head to head.
struct LaneTurn {
  f32x2 A[4], B[4];
  uint32_t mask;  // 0 in a lane past rotary_dim, whose B = 0 must not meet an infinity; else all ones
  int partner;    // the lane (of 16) of the pairs' other halves
  bool whole;     // every lane is rotated
  bool norm;
  float eps;
};

// n rows of two tokens, one a half-warp, src_step elements apart. kTurn: norm and
// rotation (kFar: pairs (i, i + rotary_dim / 2); else (2i, 2i + 1)). kE4m3: to rows of codes and
// their scales, dst_step in rows; else in elements.
template <typename T, bool kTurn, bool kFar, bool kE4m3>
__device__ inline void append_rows(const T* src, int64_t src_step, void* dst_, float* scale, int64_t dst_step, int n,
                                   bool live, int e, const LaneTurn& t, uint4* ring) {
  using Raw = Raw8<T>;
  constexpr int kPieces = Raw::kWords / 4;
  using Out = typename std::conditional<kE4m3, uint8_t, T>::type;
  Out* dst = static_cast<Out*>(dst_);
  if (kE4m3) dst_step *= kHeadDim;
  const int mine = live ? n : 0;
  auto ask = [&](int h) {  // row h into its place of the ring, one group of copies a row
    if (h < mine)
#pragma unroll
      for (int i = 0; i < kPieces; ++i)  // piece e + 16 i of the half-warp's row: whole sectors
        cp_async16(ring + (h % Raw::kAhead) * 32 * kPieces + e + 16 * i, reinterpret_cast<const uint4*>(src) + 16 * i);
    src += src_step;
    cp_async_commit();
  };
#pragma unroll
  for (int h = 0; h < Raw::kAhead; ++h) ask(h);
#pragma unroll 2
  for (int h = 0; h < n; ++h) {
    cp_async_wait<Raw::kAhead - 1>();
    if (kPieces > 1) __syncwarp();  // pieces that other lanes copied (bf16: a lane's own)
    Raw raw;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const uint4 v = ring[(h % Raw::kAhead) * 32 * kPieces + kPieces * e + i];
      raw.w[4 * i] = v.x; raw.w[4 * i + 1] = v.y; raw.w[4 * i + 2] = v.z; raw.w[4 * i + 3] = v.w;
    }
    f32x2 x[4];
    raw.unpack(x);
    if (kTurn) {
      f32x2 sq = mul2(x[0], x[0]);
#pragma unroll
      for (int j = 1; j < 4; ++j) sq = fma2(x[j], x[j], sq);
      float ss, hi;
      unpack2(sq, ss, hi);
      ss += hi;
#pragma unroll
      for (int off = 1; off < 16; off <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
      const float r = t.norm ? rsqrtf(fmaf(ss, 1.f / kHeadDim, t.eps)) : 1.f;
      Raw other;
#pragma unroll
      for (int j = 0; j < Raw::kWords; ++j)
        other.w[j] = kFar ? __shfl_sync(0xffffffffu, raw.w[j], t.partner, 16) : raw.w[j];
      if (!t.whole)
#pragma unroll
        for (int j = 0; j < Raw::kWords; ++j) other.w[j] &= t.mask;
      f32x2 y[4];
      other.unpack(y);
      const f32x2 rr = pack2(r, r);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (!kFar) {
          float lo, up;
          unpack2(y[j], lo, up);
          y[j] = pack2(up, lo);
        }
        x[j] = mul2(rr, fma2(y[j], t.B[j], mul2(x[j], t.A[j])));
      }
    }
    if (kPieces > 1) __syncwarp();
    ask(h + Raw::kAhead);
    if constexpr (kE4m3) {
      float f[8], mx = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        unpack2(x[j], f[2 * j], f[2 * j + 1]);
        mx = fmaxf(mx, fmaxf(fabsf(f[2 * j]), fabsf(f[2 * j + 1])));
      }
#pragma unroll
      for (int off = 1; off < 16; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
      mx = fmaxf(mx, kMinRowMax);
      const float inv = __fdiv_rn(kE4m3Max, mx);
      uint32_t c[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        c[j] = __nv_cvt_float2_to_fp8x2(make_float2(f[2 * j] * inv, f[2 * j + 1] * inv), __NV_SATFINITE, __NV_E4M3);
      if (live) {
        *reinterpret_cast<uint2*>(dst) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
        if (e == 0) *scale = __fdiv_rn(mx, kE4m3Max);
      }
      scale += dst_step / kHeadDim;
    } else if (live) {
      Raw::store(dst, x);
    }
    dst += dst_step;
  }
}

// A and B of a lane's eight dims: the norm weights (w null: none) times the cosines
// and sines of the token's angles (lane (e), half: lanes of one half of the rotated dims).
template <typename T, bool kFar>
__device__ inline void make_turn(LaneTurn& t, const T* w, float offset, const float2* turn, bool rot, int half, int e) {
  float wv[8], wp[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) wv[j] = wp[j] = 1.f;
  if (w != nullptr) {
    Raw8<T> r;
    r.load(w + 8 * e);
    unpack8(r, wv);
    r.load(w + 8 * t.partner);
    unpack8(r, wp);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      wv[j] += offset;
      wp[j] += offset;
    }
  }
  float pa[8], pb[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const bool first = kFar ? e < half : !(j & 1);  // the first of a pair takes -sin
    const float2 cs = rot ? turn[kFar ? 8 * (e < half ? e : e - half) + j : 4 * e + j / 2] : make_float2(1.f, 0.f);
    pa[j] = wv[j] * cs.x;
    pb[j] = wp[kFar ? j : j ^ 1] * (first ? -cs.y : cs.y);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    t.A[j] = pack2(pa[2 * j], pa[2 * j + 1]);
    t.B[j] = pack2(pb[2 * j], pb[2 * j + 1]);
  }
}

// kE4m3: keys and values go to e4m3 rows with scales. CTA: token pair blockIdx.x /
// parts, heads [u0, u0 + run) of [queries | keys | values].
template <typename T, bool kFar, bool kE4m3>
__global__ void __launch_bounds__(kAppendThreads, 8) append_kernel(AppendArgs a, int run, int parts) {
  __shared__ float2 turn[2][kHeadDim / 2];  // cos, sin of the two tokens' angles
  __shared__ uint4 rows[kAppendWarps][Raw8<T>::kAhead * Raw8<T>::kWords / 4 * 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e = lane & 15;
  uint4* ring = rows[warp] + (lane >> 4) * (Raw8<T>::kWords * 4);  // the half-warp's row in each place
  const int64_t pair = blockIdx.x / parts;
  const int nq = a.q.data != nullptr ? a.hq : 0, nk = a.k.data != nullptr ? a.hkv : 0;
  const int u0 = (blockIdx.x - static_cast<int>(pair) * parts) * run, u1 = min(u0 + run, nq + 2 * nk);
  const int rd = a.cfg.rotary_dim;
  pdl_wait();
  pdl_trigger();
  if (u0 < nq + nk && static_cast<int>(threadIdx.x & 63) < rd / 2) {
    const int i = threadIdx.x & 63;
    const int64_t token = pair * 2 + (threadIdx.x >> 6);
    const float f = a.inv_freq[i];
    float c = 1.f, s = 0.f;
    if (token < a.n_tokens) {
      const uint64_t phase = turns_per_token(f) * static_cast<uint64_t>(static_cast<int64_t>(a.positions[token]));
      // signed fraction of a turn, as half turns in [-1, 1)
      sincospif(static_cast<float>(static_cast<int32_t>(phase >> 32)) * 4.656612873077393e-10f, &s, &c);
      if (!(fabsf(f) <= 3.4028235e38f)) c = s = __int_as_float(0x7fc00000);  // not a frequency
    }
    turn[threadIdx.x >> 6][i] = make_float2(c, s);
  }

  const int64_t token = pair * 2 + (lane >> 4);
  bool live = token < a.n_tokens;
  int64_t row0 = 0;  // cache row of head 0
  if (live && a.slots != nullptr) {
    const int64_t slot = a.slots[token];
    if (slot < 0 || slot >= a.n_runs * a.cache_rows_per_head) {
      live = false;  // padding (-1), or outside the cache: nothing of the token is read or written
      if (slot != -1) set_status(a.status, MSA_ERR_DEVICE_BOUNDS, kIdAppend);
    } else {
      const int64_t r = a.cache_rows_per_head == kBlock ? slot / kBlock : slot / a.cache_rows_per_head;
      row0 = r * a.hkv * a.cache_rows_per_head + (slot - r * a.cache_rows_per_head);
    }
  }
  LaneTurn t;
  const int half = rd >> 4;  // lanes of one half of the rotated dims
  const bool rot = 8 * e < rd;
  t.partner = kFar && rot ? (e < half ? e + half : e - half) : e;
  t.mask = rot ? 0xffffffffu : 0u;
  t.whole = rd == kHeadDim;
  t.eps = a.cfg.eps;
  __syncthreads();

#pragma unroll
  for (int kind = 0; kind < 3; ++kind) {  // queries, keys, values
    const int base = kind == 0 ? 0 : kind == 1 ? nq : nq + nk;
    const int h0 = max(u0 - base, 0) + warp, h1 = min(u1 - base, kind == 0 ? nq : nk);
    if (h0 >= h1) continue;
    const int n = (h1 - h0 + kAppendWarps - 1) / kAppendWarps;  // heads h0, h0 + 4, ...
    const msa_rows& in = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
    const T* src = static_cast<const T*>(in.data) + (16 / sizeof(T)) * e;  // this lane's first piece
    if (live) src += token * in.token_stride + h0 * in.head_stride;
    const int64_t src_step = kAppendWarps * in.head_stride;
    if (kind != 2) {
      t.norm = (a.cfg.norm & (kind + 1)) != 0;
      const T* w = static_cast<const T*>(kind == 0 ? a.q_weight : a.k_weight);
      make_turn<T, kFar>(t, t.norm ? w : nullptr, a.cfg.weight_offset, turn[lane >> 4], rot, half, e);
    }
    if (kind == 0) {
      T* dst = static_cast<T*>(const_cast<void*>(a.q_out.data)) + 8 * e;
      if (live) dst += token * a.q_out.token_stride + h0 * a.q_out.head_stride;
      append_rows<T, true, kFar, false>(src, src_step, dst, nullptr, kAppendWarps * a.q_out.head_stride, n, live, e, t,
                                        ring);
      continue;
    }
    const int64_t row = row0 + h0 * a.cache_rows_per_head, step = kAppendWarps * a.cache_rows_per_head;
    void* cache = kind == 1 ? a.kc : a.vc;
    if constexpr (kE4m3) {
      float* scale = (kind == 1 ? a.k_scale : a.v_scale) + row;
      uint8_t* dst = static_cast<uint8_t*>(cache) + row * kHeadDim + 8 * e;
      if (kind == 1) append_rows<T, true, kFar, true>(src, src_step, dst, scale, step, n, live, e, t, ring);
      else append_rows<T, false, kFar, true>(src, src_step, dst, scale, step, n, live, e, t, ring);
    } else {
      T* dst = static_cast<T*>(cache) + row * kHeadDim + 8 * e;
      if (kind == 1) append_rows<T, true, kFar, false>(src, src_step, dst, nullptr, step * kHeadDim, n, live, e, t, ring);
      else append_rows<T, false, kFar, false>(src, src_step, dst, nullptr, step * kHeadDim, n, live, e, t, ring);
    }
  }
}

template <typename T, bool kE4m3>
cudaError_t launch(const AppendArgs& a, int run, int parts, unsigned grid, cudaStream_t stream) {
  if (a.cfg.interleaved)
    return launch_overlapped(append_kernel<T, false, kE4m3>, grid, kAppendThreads, 0, stream, a, run, parts);
  return launch_overlapped(append_kernel<T, true, kE4m3>, grid, kAppendThreads, 0, stream, a, run, parts);
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a, int dtype, cudaStream_t stream) {
  const int64_t units = (a.q.data != nullptr ? a.hq : 0) + (a.k.data != nullptr ? 2 * a.hkv : 0);
  const int64_t pairs = (static_cast<int64_t>(a.n_tokens) + 1) / 2;
  // A pair's heads are split over as many CTAs as it takes to give every SM
  // kCtasPerSm of them, four heads a CTA at least.
  constexpr int64_t kCtasPerSm = 4;
  int64_t parts = (kCtasPerSm * a.num_sms + pairs - 1) / pairs;
  int64_t run = (units + parts - 1) / parts;
  run = (run + kAppendWarps - 1) / kAppendWarps * kAppendWarps;
  parts = (units + run - 1) / run;
  if (pairs * parts > INT32_MAX) return cudaErrorInvalidConfiguration;
  const unsigned grid = static_cast<unsigned>(pairs * parts);
  const int r = static_cast<int>(run), p = static_cast<int>(parts);
  if (dtype == MSA_DTYPE_F32) return launch<float, false>(a, r, p, grid, stream);
  if (dtype == MSA_DTYPE_E4M3) return launch<__nv_bfloat16, true>(a, r, p, grid, stream);
  return launch<__nv_bfloat16, false>(a, r, p, grid, stream);
}

}  // namespace msa
