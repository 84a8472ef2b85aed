// What the kernels that attend over an e4m3 cache share: softmax attention of the G query heads of
// a GQA group over the listed (or all) blocks of K and V rows kept as 8-bit
// codes with one fp32 scale per row (K[t] = ks_t kc_t, V[t] = vs_t vc_t):
//   s_t = scale ks_t (q . kc_t),  l = sum_t 2^(s_t - m),
//   O = sum_t 2^(s_t + log2 vs_t - M) vc_t,  out = O 2^(M - m) / l
// (scores in log2 units). Codes go to the tensor cores as fp16, which holds
// every e4m3 value exactly; a row's scale never touches its codes: K's
// multiplies the fp32 score, V's joins the exponent of the weight, so a weight is
// one exp2 and lies below 2^kWeightGrow whatever the sizes of the rows. M is the largest
// s_t + log2 vs_t seen when it last moved, m the same of s_t (they move once a token passes them
// by kWeightGrow or kSumGrow): two references, because a row that decides l need not decide O.
//
// Rounding: a query head is scaled by a power of two to below 1 and kept in
// fp16 (11 bits: a bf16 query is exact down to 2^-16 of the head's largest element,
// and within 2^-25 of that element below). Weights are fp16 (half a step: 2^-11
// relative, 2^-8 for bf16 ones), scaled by 2^kWeightBits so that those down to
// 2^-24 of the largest keep their 11 bits and vanish only below 2^-35.
// l, O and the scores are fp32.
//
// No transpose is stored anywhere. A lane reads K and V in 16-byte pieces and the
// order of a product's terms is chosen so that those are fragments already:
//   S = K Q^T, step (hlf, w) of 8: lane (g, c) holds dims 16 (c + 4 hlf) + 4w + {0,
//     1 | 2, 3} of its two rows (the fragment's k = 2c, 2c + 1 | 2c + 8, 2c + 9),
//     Q's fragment takes the same dims.
//   O^T = V^T P^T, tile 2w + u of 8: fragment rows g, g + 8 are dims 16g + 4w + 2u
//     + {0, 1}, k = tokens; two byte permutes of the words of two tokens give
//     the pairs of one dim.
// Row g of S is token tok(g) = g ^ ((g & 1) << 2): with the 128-byte swizzle the 8
// lanes of a shared-memory phase then read 8 different 16-byte columns, of K (rows
// g, g + 1; chunks c) as of V (rows 2c; chunks g, g + 1).
#pragma once

#include <cuda_fp16.h>

#include "decode_tail.cuh"

namespace msa {

constexpr int kE8Group = 4;      // consumer warps that share a block
constexpr int kE8Consumers = 8;  // two groups
constexpr int kE8Tile = 8192;                          // 64 rows of 128 codes
constexpr int kE8ScaleBytes = kBlock * 4;              // one tile's scales
constexpr int kE8StageBytes = 2 * (kE8Tile + kE8ScaleBytes);
constexpr int kWeightBits = 10;
constexpr float kWeightGrow = 5.f;   // a weight may grow past M by this much (2^15 in fp16) before M moves
constexpr float kSumGrow = 20.f;     // and a term of l past m by this much
constexpr float kNoRef = -1.7e38f;   // M or m before any token: 2^(-inf - kNoRef) is 0
constexpr size_t kE8MergeBytes = static_cast<size_t>(kE8Group) * kMaxGroup * kHeadDim * sizeof(float);

// The producer's next blocks, looked up by its lanes.
struct E8Next {
  int64_t row[32];
  int32_t valid[32];  // tokens that exist (0: the block is skipped)
};

__device__ inline float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two e4m3 codes (low byte first) as fp16 pairs: exact.
__device__ inline void e4m3x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ inline void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                               uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ inline uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ inline uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ inline uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// A consumer warp's share of one unit: tokens [16 w, 16 w + 16) of the blocks it
// is shown, for the unit's heads (lane (g, c): heads 2c, 2c + 1).
struct E8Consumer {
  uint32_t qb[8][2];                   // Q^T fragments: head g, the dims the K fragments hold, times 2^-e
  float hs0, hs1;                      // score factors (2^e scale log2 e) of heads 2c, 2c + 1
  float M0, M1, m0, m1, l0, l1;
  float o[8][4];                       // O^T: dims 16g + 2j (0: head 2c, 1: 2c + 1) and 16g + 2j + 1 (2, 3)

  // q: the unit's grp query heads; scale_log2: the softmax scale times log2 e.
  __device__ void start(const __nv_bfloat16* q, int grp, float scale_log2, int lane) {
    const int g = lane >> 2, c = lane & 3;
    M0 = M1 = m0 = m1 = kNoRef;
    l0 = l1 = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    {
      float qf[2][16], mx = 0.f;
      const bool live = g < grp;
      const __nv_bfloat16* qrow = q + (live ? g : 0) * kHeadDim + 16 * c;
#pragma unroll
      for (int hlf = 0; hlf < 2; ++hlf)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint4 v = *reinterpret_cast<const uint4*>(qrow + 64 * hlf + 8 * i);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t x = live ? word(v, j) : 0u;
            qf[hlf][8 * i + 2 * j] = __uint_as_float(x << 16);
            qf[hlf][8 * i + 2 * j + 1] = __uint_as_float(x & 0xFFFF0000u);
          }
        }
#pragma unroll
      for (int i = 0; i < 16; ++i) mx = fmaxf(mx, fmaxf(fabsf(qf[0][i]), fabsf(qf[1][i])));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      // mx in [2^(e - 1), 2^e); e kept where 2^e and 2^-e are both normal
      const int e = min(max(static_cast<int>(__float_as_uint(mx) >> 23) - 126, -125), 125);
      const float down = __int_as_float((127 - e) << 23);
      const float up = __int_as_float((127 + e) << 23) * scale_log2;
      hs0 = __shfl_sync(0xffffffffu, up, 8 * c);      // lane (2c, 0)
      hs1 = __shfl_sync(0xffffffffu, up, 8 * c + 4);  // lane (2c + 1, 0)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float* f = &qf[k >> 2][4 * (k & 3)];
        qb[k][0] = pack_f16(f[0] * down, f[1] * down);
        qb[k][1] = pack_f16(f[2] * down, f[3] * down);
      }
    }
  }

  // The block whose K and V tiles lie at kb and kb + kE8Tile in shared memory,
  // their scales at ks and ks + kBlock; tokens [valid, 64) do not exist.
  __device__ void block(uint32_t kb, const float* ks, int valid, int w16, int lane) {
    const int g = lane >> 2, c = lane & 3;
    const uint32_t vt = kb + kE8Tile;
    const float* vs = ks + kBlock;
    const int t0 = w16 + (g ^ ((g & 1) << 2)), t1 = t0 + 8;           // tokens of S rows g, g + 8
    const int va = w16 + 2 * c, vb = w16 + ((2 * c + 1) ^ 4);         // tokens of k = 2c, 2c + 1; + 8 the others
    const uint32_t kofs0 = swz128(t0, c), kofs1 = swz128(t0, c + 4);  // row t1 is 1024 bytes on
    const uint32_t vofs0 = swz128(va, g), vofs1 = swz128(vb, g);
    const uint4 k00 = lds128(kb + kofs0), k10 = lds128(kb + kofs0 + 1024);
    const uint4 k01 = lds128(kb + kofs1), k11 = lds128(kb + kofs1 + 1024);
    uint4 v0 = lds128(vt + vofs0), v1 = lds128(vt + vofs1);
    uint4 v2 = lds128(vt + vofs0 + 1024), v3 = lds128(vt + vofs1 + 1024);
    const float ks0 = ks[t0], ks1 = ks[t1], lv0 = __log2f(vs[t0]), lv1 = __log2f(vs[t1]);
    float sa[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      uint32_t a0, a1, a2, a3;
      e4m3x4_to_f16(word(k00, w), a0, a2);
      e4m3x4_to_f16(word(k10, w), a1, a3);
      mma_f16(sa, a0, a1, a2, a3, qb[w][0], qb[w][1]);
      e4m3x4_to_f16(word(k01, w), a0, a2);
      e4m3x4_to_f16(word(k11, w), a1, a3);
      mma_f16(sb, a0, a1, a2, a3, qb[4 + w][0], qb[4 + w][1]);
    }
    float s0 = (sa[0] + sb[0]) * ks0 * hs0, s1 = (sa[1] + sb[1]) * ks0 * hs1;  // token t0, heads 2c, 2c + 1
    float s2 = (sa[2] + sb[2]) * ks1 * hs0, s3 = (sa[3] + sb[3]) * ks1 * hs1;  // token t1
    float x0 = s0 + lv0, x1 = s1 + lv0, x2 = s2 + lv1, x3 = s3 + lv1;
    if (valid < kBlock) {  // tokens past the end: whatever their rows and scales hold
      if (t0 >= valid) s0 = s1 = x0 = x1 = -INFINITY;
      if (t1 >= valid) s2 = s3 = x2 = x3 = -INFINITY;
      const uint4 none = make_uint4(0u, 0u, 0u, 0u);
      if (va >= valid) v0 = none;
      if (vb >= valid) v1 = none;
      if (va + 8 >= valid) v2 = none;
      if (vb + 8 >= valid) v3 = none;
    }
    const float sm0 = fmaxf(s0, s2), sm1 = fmaxf(s1, s3);
    float xm0 = fmaxf(x0, x2), xm1 = fmaxf(x1, x3);
    const bool move = xm0 > M0 + kWeightGrow || xm1 > M1 + kWeightGrow || sm0 > m0 + kSumGrow ||
                      sm1 > m1 + kSumGrow;
    if (__any_sync(0xffffffffu, move)) {
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        xm0 = fmaxf(xm0, __shfl_xor_sync(0xffffffffu, xm0, off));
        xm1 = fmaxf(xm1, __shfl_xor_sync(0xffffffffu, xm1, off));
      }
      const float n0 = fmaxf(M0, xm0), n1 = fmaxf(M1, xm1);  // shared by the lanes of a head
      const float f0 = ex2(M0 - n0), f1 = ex2(M1 - n1);
      M0 = n0;
      M1 = n1;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        o[j][0] *= f0; o[j][1] *= f1; o[j][2] *= f0; o[j][3] *= f1;
      }
      const float p0 = fmaxf(m0, sm0), p1 = fmaxf(m1, sm1);  // each lane's own
      l0 *= ex2(m0 - p0);
      l1 *= ex2(m1 - p1);
      m0 = p0;
      m1 = p1;
    }
    l0 += ex2(s0 - m0) + ex2(s2 - m0);
    l1 += ex2(s1 - m1) + ex2(s3 - m1);
    const float r0 = M0 - kWeightBits, r1 = M1 - kWeightBits;
    const uint32_t pb0 = movm_t(pack_f16(ex2(x0 - r0), ex2(x1 - r1)));  // k = 2c, 2c + 1 of head g
    const uint32_t pb1 = movm_t(pack_f16(ex2(x2 - r0), ex2(x3 - r1)));
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      uint32_t a0, a1, a2, a3;
      e4m3x4_to_f16(__byte_perm(word(v0, w), word(v1, w), 0x5140), a0, a1);
      e4m3x4_to_f16(__byte_perm(word(v2, w), word(v3, w), 0x5140), a2, a3);
      mma_f16(o[2 * w], a0, a1, a2, a3, pb0, pb1);
      e4m3x4_to_f16(__byte_perm(word(v0, w), word(v1, w), 0x7362), a0, a1);
      e4m3x4_to_f16(__byte_perm(word(v2, w), word(v3, w), 0x7362), a2, a3);
      mma_f16(o[2 * w + 1], a0, a1, a2, a3, pb0, pb1);
    }
  }

  // One m and l for the 8 lanes that share c, and O relative to that m.
  __device__ void finish() {
    float a0 = m0, a1 = m1;
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      a0 = fmaxf(a0, __shfl_xor_sync(0xffffffffu, a0, off));
      a1 = fmaxf(a1, __shfl_xor_sync(0xffffffffu, a1, off));
    }
    l0 *= ex2(m0 - a0);
    l1 *= ex2(m1 - a1);
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, off);
      l1 += __shfl_xor_sync(0xffffffffu, l1, off);
    }
    const float f0 = exp2f(M0 - kWeightBits - a0), f1 = exp2f(M1 - kWeightBits - a1);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      o[j][0] *= f0; o[j][1] *= f1; o[j][2] *= f0; o[j][3] *= f1;
    }
    m0 = a0 == kNoRef ? -INFINITY : a0;
    m1 = a1 == kNoRef ? -INFINITY : a1;
    // a NaN among the scores never moved m: keep it visible to the merge
    if (l0 != l0) m0 = 0.f;
    if (l1 != l1) m1 = 0.f;
  }

  // Joins the eight warps' states (all consumers call it, after finish()): the
  // second group hands its registers to the first lane by lane, whose four states
  // go to `buf` (kE8MergeBytes) head by head, where warp w takes head w and lane
  // l of it dims 4l .. 4l + 3. A pair of dims (16g + 2j, + 1) is kept at 16g + 2 ((j
  // + g) mod 8), so that the eight g of a store meet different banks. `free`: run
  // by each warp once its own state is handed over (by the second group while the
  // first joins). A call's buffers may be used again by the call after the next.
  template <typename F>
  __device__ void merge(float* buf, float (*wm)[kMaxGroup], float (*wl)[kMaxGroup], int warp, int lane, F free,
                        float& M, float& L, float4& acc) {
    const int g = lane >> 2, c = lane & 3;
    float* mine = buf + (warp & 3) * kMaxGroup * kHeadDim;
    if (warp >= kE8Group) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        reinterpret_cast<float4*>(mine)[j * 32 + lane] = make_float4(o[j][0], o[j][1], o[j][2], o[j][3]);
      hand_over(wm[warp], wl[warp], g, c);
      bar_arrive_warps(1, 32 * kE8Consumers);
      free();
    } else {
      bar_sync_warps(1, 32 * kE8Consumers);
      const float* pm = wm[warp + kE8Group];
      const float* pl = wl[warp + kE8Group];
      const float pm0 = pm[2 * c], pm1 = pm[2 * c + 1];
      const float t0 = fmaxf(m0, pm0), t1 = fmaxf(m1, pm1);
      const float r0 = t0 == -INFINITY ? 0.f : t0, r1 = t1 == -INFINITY ? 0.f : t1;
      const float fa0 = ex2(m0 - r0), fb0 = ex2(pm0 - r0), fa1 = ex2(m1 - r1), fb1 = ex2(pm1 - r1);
      l0 = l0 * fa0 + pl[2 * c] * fb0;
      l1 = l1 * fa1 + pl[2 * c + 1] * fb1;
      m0 = t0;
      m1 = t1;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float4 v = reinterpret_cast<const float4*>(mine)[j * 32 + lane];
        o[j][0] = fmaf(v.x, fb0, o[j][0] * fa0);
        o[j][1] = fmaf(v.y, fb1, o[j][1] * fa1);
        o[j][2] = fmaf(v.z, fb0, o[j][2] * fa0);
        o[j][3] = fmaf(v.w, fb1, o[j][3] * fa1);
      }
      __syncwarp();
      float* row = mine + 2 * c * kHeadDim + 16 * g;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int at = 2 * ((j + g) & 7);
        *reinterpret_cast<float2*>(row + at) = make_float2(o[j][0], o[j][2]);
        *reinterpret_cast<float2*>(row + kHeadDim + at) = make_float2(o[j][1], o[j][3]);
      }
      hand_over(wm[warp], wl[warp], g, c);
    }
    bar_sync_warps(2, 32 * kE8Consumers);
    M = fmaxf(fmaxf(wm[0][warp], wm[1][warp]), fmaxf(wm[2][warp], wm[3][warp]));
    const float ref = M == -INFINITY ? 0.f : M;
    const int gg = lane >> 2, j0 = 2 * (lane & 3);
    const float* col = buf + warp * kHeadDim + 16 * gg;
    const int at0 = 2 * ((j0 + gg) & 7), at1 = 2 * ((j0 + 1 + gg) & 7);
    L = 0.f;
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kE8Group; ++i) {
      const float f = ex2(wm[i][warp] - ref);
      const float2 a = *reinterpret_cast<const float2*>(col + i * kMaxGroup * kHeadDim + at0);
      const float2 b = *reinterpret_cast<const float2*>(col + i * kMaxGroup * kHeadDim + at1);
      L = fmaf(f, wl[i][warp], L);
      acc.x = fmaf(f, a.x, acc.x);
      acc.y = fmaf(f, a.y, acc.y);
      acc.z = fmaf(f, b.x, acc.z);
      acc.w = fmaf(f, b.y, acc.w);
    }
    if (warp < kE8Group) free();
  }
  __device__ void hand_over(float (&wm)[kMaxGroup], float (&wl)[kMaxGroup], int g, int c) const {
    if (g != 0) return;
    wm[2 * c] = m0;
    wm[2 * c + 1] = m1;
    wl[2 * c] = l0;
    wl[2 * c + 1] = l1;
  }
};

// Issues one block's copies (one thread); `valid` 0: a block to be skipped.
__device__ inline void e8_issue(const CUtensorMap* tmk, const CUtensorMap* tmv, const float* k_scale,
                                const float* v_scale, int64_t row, int valid, uint8_t* tiles, uint8_t* scales,
                                int32_t* stage_valid, uint64_t* full) {
  *stage_valid = valid;
  if (valid == 0) {
    mbar_arrive(full);
    return;
  }
  mbar_arrive_expect_tx(full, kE8StageBytes);
  tma_load_2d(tiles, tmk, 0, static_cast<int32_t>(row), full);
  bulk_load(scales, k_scale + row, kE8ScaleBytes, full);
  tma_load_2d(tiles + kE8Tile, tmv, 0, static_cast<int32_t>(row), full);
  bulk_load(scales + kE8ScaleBytes, v_scale + row, kE8ScaleBytes, full);
}

// The producer warp: blocks 0 .. n - 1 of a CTA into its ring of S stages. The lanes
// look up 32 blocks at a time (find(i, row, valid): the list entry, the page),
// which would cost a chain of memory latencies one by one; lane 0 issues them.
template <int S, typename Find>
__device__ inline void e8_produce(const CUtensorMap* tmk, const CUtensorMap* tmv, const float* k_scale,
                                  const float* v_scale, int n, uint8_t* ring, uint8_t* scales, uint64_t* full,
                                  uint64_t* empty, int32_t* stage_valid, E8Next& next, int32_t* status, int lane,
                                  Find find) {
  int issued = 0;
  bool ok = true;
  for (int base = 0; base < n && ok; base += 32) {
    if (base + lane < n) find(base + lane, next.row[lane], next.valid[lane]);
    __syncwarp();
    if (lane == 0) {
      const int m = min(32, n - base);
      for (int j = 0; j < m; ++j) {
        const int stg = issued % S;
        if (issued >= S && !mbar_wait(&empty[stg], ((issued / S) - 1) & 1, status, kIdDecode)) {
          ok = false;
          break;
        }
        ++issued;
        e8_issue(tmk, tmv, k_scale, v_scale, next.row[j], next.valid[j], ring + stg * 2 * kE8Tile,
                 scales + stg * 2 * kE8ScaleBytes, &stage_valid[stg], &full[stg]);
      }
    }
    ok = __shfl_sync(0xffffffffu, ok, 0);
  }
  if (lane == 0) mbar_drain(full, S, issued, status, kIdDecode);
}

// Row and number of existing tokens of logical block `blk` of (s, h), -1 and 0 for
// one to be skipped: none (-1), past the sequence or on a bad page (both reported).
__device__ inline void e8_find(const KvView& kv, int s, int h, int64_t blk, int64_t tokens, int32_t* status,
                               int64_t& row, int32_t& valid) {
  row = -1;
  if (blk * kBlock >= tokens) set_status(status, MSA_ERR_DEVICE_BOUNDS, kIdDecode);
  else if (blk >= 0) row = kv.block_row(s, h, blk, status, kIdDecode);
  valid = row < 0 ? 0 : static_cast<int32_t>(min(static_cast<int64_t>(kBlock), tokens - blk * kBlock));
}

}  // namespace msa
