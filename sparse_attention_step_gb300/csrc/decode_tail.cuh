// What the decode attention kernels share: the CTA's block list, the merge of
// its consumer warps' softmax states and the split-K combine.
#pragma once

#include <float.h>

#include "kernels.cuh"

namespace msa {

constexpr int kMaxGroup = 8;           // query heads per KV head handled per CTA
constexpr int kMaxListPerCta = 512;    // selected blocks handled by one CTA
constexpr int kPartFloats = 2 * kMaxGroup + kMaxGroup * kHeadDim;  // m[8], l[8], o[8][128]
constexpr int kOStride = kHeadDim + 4;  // padded row of the merge buffer
constexpr int kMaxSplits = 256;         // CTAs per unit (split-K)

// Shared memory of one CTA with NW consumer warps (after the 1024-aligned
// stage ring).
template <int NW>
struct DecodeTail {
  uint64_t full[8];
  uint64_t empty[8];
  int32_t blocks[kMaxListPerCta];
  int32_t n_blocks;
  int32_t dense_lo;  // dense: block i of this CTA is dense_lo + i (no list)
  int32_t is_last;
  float wm[NW][kMaxGroup];
  float wl[NW][kMaxGroup];
};

// Writes the per-warp state into the merge buffer (rows = heads, padded).
// Then merges `nw` states -> (M, L, O) for head/dims owned by this thread.
__device__ inline void merge_states(int nw, const float* wm, const float* wl, int wstride, const float* o,
                                    int ostride_w, int head, int d0, float& M, float& L, float (&acc)[8]) {
  M = -INFINITY;
  for (int w = 0; w < nw; ++w) M = fmaxf(M, wm[w * wstride + head]);
  L = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.f;
  if (M == -INFINITY) return;
  for (int w = 0; w < nw; ++w) {
    const float f = exp2f(wm[w * wstride + head] - M);
    L += f * wl[w * wstride + head];
    const float* src = o + w * ostride_w + head * kOStride + d0;
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = fmaf(f, src[i], acc[i]);
  }
}

template <typename T>
__device__ inline void store_out8(T* dst, const float (&x)[8]);
template <>
__device__ inline void store_out8<__nv_bfloat16>(__nv_bfloat16* dst, const float (&x)[8]) {
  uint4 o;
  o.x = pack_bf16(x[0], x[1]);
  o.y = pack_bf16(x[2], x[3]);
  o.z = pack_bf16(x[4], x[5]);
  o.w = pack_bf16(x[6], x[7]);
  *reinterpret_cast<uint4*>(dst) = o;
}
template <>
__device__ inline void store_out8<float>(float* dst, const float (&x)[8]) {
  reinterpret_cast<float4*>(dst)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(dst)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// Final normalisation of one (head, 8 dims) piece.
template <typename T>
__device__ inline void write_final(const DecodeArgs& a, int s, int h, int head, int d0, float M, float L,
                                   const float (&acc)[8]) {
  float x[8];
  const float inv = (L > 0.f) ? 1.f / L : 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = acc[i] * inv;
  const int64_t qrow = static_cast<int64_t>(s) * a.hq + h * a.grp + head;
  store_out8<T>(reinterpret_cast<T*>(a.out) + qrow * kHeadDim + d0, x);
  if (a.lse != nullptr && d0 == 0) a.lse[qrow] = lse_of(M, L);
}

// The CTA-level tail shared by both paths: merge the consumer warps' states
// (already in shared memory), then either write the output (one split) or the
// partial + ticket, with the last CTA of the unit merging all partials.
// `scratch` is free shared memory of at least 2 * kMaxGroup * n_splits + 16
// floats (the merge buffer may be reused once the warp merge is done).
template <typename T, int NW>
__device__ void decode_tail(const DecodeArgs& a, DecodeTail<NW>& st, const float* obuf, float* scratch, int s, int h,
                            int split) {
  const int tid = threadIdx.x;
  const int64_t unit = static_cast<int64_t>(s) * a.hkv + h;
  // 8 heads x 16 eight-dim pieces = 128 items; threads 0..127
  const int head = tid >> 4;
  const int d0 = (tid & 15) * 8;
  const bool worker = tid < 128 && head < a.grp;
  float M = -INFINITY, L = 0.f, acc[8];
  if (worker) merge_states(NW, &st.wm[0][0], &st.wl[0][0], kMaxGroup, obuf, kMaxGroup * kOStride, head,
                           d0, M, L, acc);
  if (a.n_splits == 1) {
    if (worker) write_final<T>(a, s, h, head, d0, M, L, acc);
    return;
  }
  float* part = a.partials + (unit * a.n_splits + split) * kPartFloats;
  if (worker) {
    if (d0 == 0) {
      part[head] = M;
      part[kMaxGroup + head] = L;
    }
    float* po = part + 2 * kMaxGroup + head * kHeadDim + d0;
    reinterpret_cast<float4*>(po)[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    reinterpret_cast<float4*>(po)[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
  }
  __threadfence();
  __syncthreads();
  if (tid == 0) {
    const int prev = atomicAdd(&a.tickets[unit], 1);
    st.is_last = (prev == a.n_splits - 1);
  }
  __syncthreads();
  if (!st.is_last) return;
  __threadfence();
  // Last CTA of the unit. (1) every (split, head) max and sum, in parallel.
  const int n = a.n_splits;
  const float* base = a.partials + unit * n * kPartFloats;
  float* fm = scratch;                        // [n][8]: max, then the scale factor 2^(m_i - M)
  float* fl = scratch + n * kMaxGroup;        // [n][8]: sums
  float* tot = scratch + 2 * n * kMaxGroup;   // [8] M, [8] L
  for (int i = tid; i < n * kMaxGroup; i += blockDim.x) {
    const int sp = i / kMaxGroup, hh = i % kMaxGroup;
    fm[i] = __ldcg(base + sp * kPartFloats + hh);
    fl[i] = __ldcg(base + sp * kPartFloats + kMaxGroup + hh);
  }
  __syncthreads();
  // (2) per head: global max, factors and total sum
  if (tid < kMaxGroup) {
    float Mx = -INFINITY;
    for (int i = 0; i < n; ++i) Mx = fmaxf(Mx, fm[i * kMaxGroup + tid]);
    float Lx = 0.f;
    for (int i = 0; i < n; ++i) {
      const float f = (Mx == -INFINITY) ? 0.f : exp2f(fm[i * kMaxGroup + tid] - Mx);
      fm[i * kMaxGroup + tid] = f;
      Lx += f * fl[i * kMaxGroup + tid];
    }
    tot[tid] = Mx;
    tot[kMaxGroup + tid] = Lx;
  }
  __syncthreads();
  // (3) weighted sum of the partial outputs, several splits in flight
  if (worker) {
    float o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = 0.f;
    const float* po = base + 2 * kMaxGroup + head * kHeadDim + d0;
    int i = 0;
    for (; i + 4 <= n; i += 4) {
      float4 u[4], v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        u[j] = __ldcg(reinterpret_cast<const float4*>(po + (i + j) * kPartFloats));
        v[j] = __ldcg(reinterpret_cast<const float4*>(po + (i + j) * kPartFloats + 4));
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float f = fm[(i + j) * kMaxGroup + head];
        o[0] = fmaf(f, u[j].x, o[0]); o[1] = fmaf(f, u[j].y, o[1]); o[2] = fmaf(f, u[j].z, o[2]);
        o[3] = fmaf(f, u[j].w, o[3]); o[4] = fmaf(f, v[j].x, o[4]); o[5] = fmaf(f, v[j].y, o[5]);
        o[6] = fmaf(f, v[j].z, o[6]); o[7] = fmaf(f, v[j].w, o[7]);
      }
    }
    for (; i < n; ++i) {
      const float4 u = __ldcg(reinterpret_cast<const float4*>(po + i * kPartFloats));
      const float4 v = __ldcg(reinterpret_cast<const float4*>(po + i * kPartFloats + 4));
      const float f = fm[i * kMaxGroup + head];
      o[0] = fmaf(f, u.x, o[0]); o[1] = fmaf(f, u.y, o[1]); o[2] = fmaf(f, u.z, o[2]); o[3] = fmaf(f, u.w, o[3]);
      o[4] = fmaf(f, v.x, o[4]); o[5] = fmaf(f, v.y, o[5]); o[6] = fmaf(f, v.z, o[6]); o[7] = fmaf(f, v.w, o[7]);
    }
    write_final<T>(a, s, h, head, d0, tot[head], tot[kMaxGroup + head], o);
  }
  if (tid == 0) a.tickets[unit] = 0;  // ready for the next call
}

// Split-K combine inside a thread-block cluster (the unit's n_splits CTAs, n a
// power of two <= 16), each CTA's merged state in `xch` (M[8], L[8],
// O[8][128]): after a cluster barrier, CTA r produces the output pieces
// r, r + n, ... (a piece = 8 dims of one head) by reading every CTA's `xch`
// through distributed shared memory, one source per lane of an n-lane group,
// reduced with shuffles. A second barrier keeps each `xch` alive until read.
template <typename T>
__device__ void cluster_join(const DecodeArgs& a, const float* xch, int s, int h) {
  const int tid = threadIdx.x;
  cluster_sync();
  if (tid < 128) {
    const int n = a.n_splits;
    const uint32_t r = cluster_ctarank();
    const int pieces = a.grp * 16;
    const int j = tid / n, i = tid % n;
    const int piece = j * n + static_cast<int>(r);
    const bool live = piece < pieces;
    const int head = live ? piece >> 4 : 0;
    const int d0 = live ? (piece & 15) * 8 : 0;
    float Mi = -INFINITY, Li = 0.f;
    float4 oa = make_float4(0.f, 0.f, 0.f, 0.f), ob = oa;
    if (live) {
      const uint32_t base = dsmem_addr(smem_u32(xch), static_cast<uint32_t>(i));
      Mi = ld_dsmem(base + 4u * head);
      Li = ld_dsmem(base + 4u * (kMaxGroup + head));
      oa = ld_dsmem4(base + 4u * (2 * kMaxGroup + head * kHeadDim + d0));
      ob = ld_dsmem4(base + 4u * (2 * kMaxGroup + head * kHeadDim + d0 + 4));
    }
    float Mx = Mi;
    for (int off = n >> 1; off > 0; off >>= 1) Mx = fmaxf(Mx, __shfl_xor_sync(0xffffffffu, Mx, off));
    const float f = (Mx == -INFINITY) ? 0.f : exp2f(Mi - Mx);
    float v[9] = {f * Li, f * oa.x, f * oa.y, f * oa.z, f * oa.w, f * ob.x, f * ob.y, f * ob.z, f * ob.w};
    for (int off = n >> 1; off > 0; off >>= 1) {
#pragma unroll
      for (int q = 0; q < 9; ++q) v[q] += __shfl_xor_sync(0xffffffffu, v[q], off);
    }
    if (live && i == 0) {
      const float o[8] = {v[1], v[2], v[3], v[4], v[5], v[6], v[7], v[8]};
      write_final<T>(a, s, h, head, d0, Mx, v[0], o);
    }
  }
  cluster_sync();
}

// The cluster tail of a CTA whose warps' states are in `obuf`: merged into
// `xch`, then joined.
template <typename T, int NW>
__device__ void decode_tail_cluster(const DecodeArgs& a, DecodeTail<NW>& st, const float* obuf, float* xch, int s,
                                    int h) {
  const int tid = threadIdx.x;
  {
    const int head = tid >> 4;
    const int d0 = (tid & 15) * 8;
    if (tid < 128 && head < a.grp) {
      float M, L, acc[8];
      merge_states(NW, &st.wm[0][0], &st.wl[0][0], kMaxGroup, obuf, kMaxGroup * kOStride, head, d0, M, L,
                   acc);
      if (d0 == 0) {
        xch[head] = M;
        xch[kMaxGroup + head] = L;
      }
      float* dst = xch + 2 * kMaxGroup + head * kHeadDim + d0;
      reinterpret_cast<float4*>(dst)[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
      reinterpret_cast<float4*>(dst)[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
    }
  }
  cluster_join<T>(a, xch, s, h);
}

// Collects this CTA's list of valid blocks into shared memory (warp 0: one
// entry per lane, compacted with a ballot).
template <int NW>
__device__ inline void gather_block_list(const DecodeArgs& a, const KvView& kv, DecodeTail<NW>& st, int s, int h,
                                         int split, int64_t nb) {
  const int tid = threadIdx.x;
  if (tid >= 32) return;
  const int lane = tid;
  int n = 0;
  if (a.idx != nullptr) {
    const int32_t* list = a.idx + (static_cast<int64_t>(s) * a.hkv + h) * a.k_total;
    const int lo = split * a.bps;
    const int hi = min(a.k_total, lo + a.bps);
    for (int base = lo; base < hi; base += 32) {
      const int i = base + lane;
      const int32_t b = i < hi ? list[i] : -1;
      if (b >= nb) set_status(a.status, MSA_ERR_DEVICE_BOUNDS, kIdDecode);
      const bool ok = b >= 0 && b < nb;
      const unsigned m = __ballot_sync(0xffffffffu, ok);
      const int at = n + __popc(m & ((1u << lane) - 1u));
      if (ok && at < kMaxListPerCta) st.blocks[at] = b;
      if (ok && at >= kMaxListPerCta) set_status(a.status, MSA_ERR_UNSUPPORTED, kIdDecode);
      n = min(n + __popc(m), kMaxListPerCta);
    }
  } else {
    const int64_t lo = static_cast<int64_t>(split) * a.bps;
    const int64_t hi = min(nb, lo + a.bps);
    n = hi > lo ? static_cast<int>(hi - lo) : 0;
    if (lane == 0) st.dense_lo = static_cast<int32_t>(lo);
  }
  if (lane == 0) st.n_blocks = n;
}

}  // namespace msa
