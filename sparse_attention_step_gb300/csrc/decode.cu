// Step 2, decode: softmax attention of the G query heads of a GQA group over
// the selected KV blocks of their group ("MiniMax goes sparse", §1 Step 2:
// the group loads one set of KV blocks and all its heads attend over it).
//
// One CTA handles a slice of one (sequence, KV head) unit's block list
// (split-K). bf16 path:
//   warp 4 (one lane) is the producer: it streams each selected 64x128 K and V
//     block into a ring of shared-memory stages with 2-D TMA copies (two
//     64-column boxes per tensor, 128-byte swizzle), one mbarrier per stage.
//   warps 0-3 are consumers: warp w owns tokens [16w, 16w+16) of every block.
//     S = K_w Q^T on tensor cores (mma m16n8k16: 16 tokens x 8 heads x 16
//     dims), online softmax per head in fp32 (exp2 with log2(e) folded into
//     the scale), then O^T += V_w^T P^T (16 dims x 8 heads x 16 tokens); P^T
//     comes from the S accumulators by an 8x8 transpose (movmatrix).
// The four warps' (m, l, O) are merged in shared memory; with several splits
// each CTA writes its partial to the workspace and the last CTA of the unit to
// finish (atomic ticket) merges them:
//   m = max_i m_i, l = sum_i l_i 2^(m_i - m), o = sum_i o_i 2^(m_i - m) / l.
// No CTA ever waits for another one.
//
// fp32 KV path: the same split/merge structure with a CUDA-core consumer
// (warp per 16 tokens, lane per 4 dims); used for fp32 caches only.
#include "decode_tail.cuh"

namespace msa {

constexpr int kDecConsumers = 4;       // consumer warps
constexpr int kDecThreads = 32 * (kDecConsumers + 1);
constexpr int kStageBytes = 4 * 8192;  // K (2 x 64x64 bf16) + V (2 x 64x64 bf16)
using DecodeSmemTail = DecodeTail<kDecConsumers>;

// ---------------------------------------------------------------------------
// bf16 kernel. grid (n_splits, Hkv, batch), kDecThreads threads.
// ---------------------------------------------------------------------------
template <int kStages>
__global__ void __launch_bounds__(kDecThreads) decode_bf16_kernel(const __grid_constant__ CUtensorMap tmk,
                                                                 const __grid_constant__ CUtensorMap tmv, KvView kv,
                                                                 DecodeArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* ring = smem_align1024(smem_raw);
  DecodeSmemTail& st = *reinterpret_cast<DecodeSmemTail*>(ring + kStages * kStageBytes);

  const int split = blockIdx.x, h = blockIdx.y, s = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&st.full[i], 1);
      mbar_init(&st.empty[i], kDecConsumers);
    }
    fence_mbar_init();
  }
  if (warp == kDecConsumers && lane == 0) {
    tma_prefetch_desc(&tmk);
    tma_prefetch_desc(&tmv);
  }
  pdl_wait();  // the index lists (and every other input) come from earlier work
  const int64_t len = kv.seq_len(s, a.status, kIdDecode);
  const int64_t nb = (len + kBlock - 1) / kBlock;
  gather_block_list(a, kv, st, s, h, split, nb);
  __syncthreads();
  const int nblk = st.n_blocks;

  const int g = lane >> 2, c = lane & 3;
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
  float o[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

  if (warp == kDecConsumers) {
    // ---------------- producer ----------------
    if (lane == 0) {
      int issued = 0;
      for (int i = 0; i < nblk; ++i) {
        const int stg = i % kStages;
        if (i >= kStages && !mbar_wait(&st.empty[stg], ((i / kStages) - 1) & 1, a.status, kIdDecode)) break;
        issued = i + 1;
        const int64_t row = kv.block_row(s, h, a.idx ? st.blocks[i] : st.dense_lo + i, a.status, kIdDecode);
        uint8_t* dst = ring + stg * kStageBytes;
        mbar_arrive_expect_tx(&st.full[stg], kStageBytes);
        const int32_t y = static_cast<int32_t>(row < 0 ? 0 : row);
        tma_load_2d(dst, &tmk, 0, y, &st.full[stg]);
        tma_load_2d(dst + 8192, &tmk, 64, y, &st.full[stg]);
        tma_load_2d(dst + 16384, &tmv, 0, y, &st.full[stg]);
        tma_load_2d(dst + 24576, &tmv, 64, y, &st.full[stg]);
      }
      mbar_drain(st.full, kStages, issued, a.status, kIdDecode);
    }
  } else {
    // ---------------- consumers ----------------
    // Q^T fragments (B operand of S = K Q^T): head g, dims 16kk + 2c (+1), +8 (+9)
    uint32_t qb[8][2];
    {
      const bool live = g < a.grp;
      const __nv_bfloat16* qrow = reinterpret_cast<const __nv_bfloat16*>(a.q) +
                                  (static_cast<int64_t>(s) * a.hq + h * a.grp + (live ? g : 0)) * kHeadDim;
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        qb[kk][0] = live ? *reinterpret_cast<const uint32_t*>(qrow + 16 * kk + 2 * c) : 0u;
        qb[kk][1] = live ? *reinterpret_cast<const uint32_t*>(qrow + 16 * kk + 2 * c + 8) : 0u;
      }
    }
    const int krow = 16 * warp + (lane & 7) + ((lane >> 3) & 1) * 8;  // K ldmatrix row
    const int kchunk = lane >> 4;
    const int vrow = 16 * warp + (lane & 7) + ((lane >> 4) & 1) * 8;  // V ldmatrix.trans row
    const int vchunk = (lane >> 3) & 1;
    for (int i = 0; i < nblk; ++i) {
      const int stg = i % kStages;
      if (!mbar_wait_warp(&st.full[stg], (i / kStages) & 1, a.status, kIdDecode)) break;
      const uint32_t kbase = smem_u32(ring + stg * kStageBytes);
      const uint32_t vbase = kbase + 16384;
      float sacc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        uint32_t a0, a1, a2, a3;
        ldsm_x4(kbase + (kk >> 2) * 8192 + swz128(krow, (kk & 3) * 2 + kchunk), a0, a1, a2, a3);
        mma_bf16(sacc, a0, a1, a2, a3, qb[kk][0], qb[kk][1]);
      }
      const int64_t first = static_cast<int64_t>(a.idx ? st.blocks[i] : st.dense_lo + i) * kBlock + 16 * warp;
      const int64_t tok = first + g;
      const bool v0 = tok < len, v1 = tok + 8 < len;
      if (first + 16 > len) {  // this warp alone reads its 16 rows of V
        const int64_t left = len - first;
        zero_tile_rows(ring + stg * kStageBytes + 16384, 8192, 16 * warp + (left > 0 ? static_cast<int>(left) : 0),
                       16 * warp + 16, lane, 32);
        __syncwarp();
      }
      const float s0 = v0 ? sacc[0] * a.scale_log2 : -INFINITY;  // token g,   head 2c
      const float s1 = v0 ? sacc[1] * a.scale_log2 : -INFINITY;  // token g,   head 2c+1
      const float s2 = v1 ? sacc[2] * a.scale_log2 : -INFINITY;  // token g+8, head 2c
      const float s3 = v1 ? sacc[3] * a.scale_log2 : -INFINITY;  // token g+8, head 2c+1
      float mx0 = fmaxf(s0, s2), mx1 = fmaxf(s1, s3);
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, off));
        mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, off));
      }
      const float mn0 = fmaxf(m0, mx0), mn1 = fmaxf(m1, mx1);
      const float r0 = mn0 == -INFINITY ? 0.f : mn0;
      const float r1 = mn1 == -INFINITY ? 0.f : mn1;
      const float al0 = exp2f(m0 - r0), al1 = exp2f(m1 - r1);
      const float p0 = exp2f(s0 - r0), p2 = exp2f(s2 - r0);
      const float p1 = exp2f(s1 - r1), p3 = exp2f(s3 - r1);
      l0 = l0 * al0 + p0 + p2;
      l1 = l1 * al1 + p1 + p3;
      m0 = mn0;
      m1 = mn1;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        o[j][0] *= al0; o[j][1] *= al1; o[j][2] *= al0; o[j][3] *= al1;
      }
      const uint32_t pb0 = movm_t(pack_bf16(p0, p1));  // tokens 0-7  -> (k = 2c.., n = head g)
      const uint32_t pb1 = movm_t(pack_bf16(p2, p3));  // tokens 8-15
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t a0, a1, a2, a3;
        ldsm_x4_t(vbase + (j >> 2) * 8192 + swz128(vrow, (j & 3) * 2 + vchunk), a0, a1, a2, a3);
        mma_bf16(o[j], a0, a1, a2, a3, pb0, pb1);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&st.empty[stg]);
    }
    // l partial sums live on the 8 lanes that share c
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, off);
      l1 += __shfl_xor_sync(0xffffffffu, l1, off);
    }
    // a NaN among the scores never moved m: keep it visible to the merge
    if (l0 != l0) m0 = 0.f;
    if (l1 != l1) m1 = 0.f;
  }
  pdl_trigger();    // the next kernel may start its set-up
  __syncthreads();  // every consumer is done with the ring: reuse it for the merge
  if (warp < kDecConsumers) {
    float* obuf = reinterpret_cast<float*>(ring) + warp * kMaxGroup * kOStride;
    if (g == 0) {
      st.wm[warp][2 * c] = m0;
      st.wm[warp][2 * c + 1] = m1;
      st.wl[warp][2 * c] = l0;
      st.wl[warp][2 * c + 1] = l1;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      obuf[(2 * c) * kOStride + 16 * j + g] = o[j][0];
      obuf[(2 * c + 1) * kOStride + 16 * j + g] = o[j][1];
      obuf[(2 * c) * kOStride + 16 * j + g + 8] = o[j][2];
      obuf[(2 * c + 1) * kOStride + 16 * j + g + 8] = o[j][3];
    }
  }
  __syncthreads();
  if (a.n_splits > 1) {
    decode_tail_cluster<__nv_bfloat16, kDecConsumers>(a, st, reinterpret_cast<const float*>(ring),
                                       reinterpret_cast<float*>(ring) + kDecConsumers * kMaxGroup * kOStride, s, h);
  } else {
    decode_tail<__nv_bfloat16, kDecConsumers>(a, st, reinterpret_cast<const float*>(ring),
                               reinterpret_cast<float*>(ring) + kDecConsumers * kMaxGroup * kOStride, s, h, split);
  }
}

// ---------------------------------------------------------------------------
// fp32 kernel (CUDA cores). grid (n_splits, Hkv, batch), kDecThreads threads;
// warps 0-3 compute, warp 4 idles until the merge.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kDecThreads) decode_f32_kernel(const float* __restrict__ k,
                                                                const float* __restrict__ v, KvView kv,
                                                                DecodeArgs a) {
  __shared__ __align__(16) float obuf[kDecConsumers * kMaxGroup * kOStride];
  __shared__ __align__(16) float merge_scratch[2 * kMaxGroup * kMaxSplits + 2 * kMaxGroup];
  __shared__ DecodeSmemTail st;
  const int split = blockIdx.x, h = blockIdx.y, s = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t len = kv.seq_len(s, a.status, kIdDecode);
  const int64_t nb = (len + kBlock - 1) / kBlock;
  gather_block_list(a, kv, st, s, h, split, nb);
  __syncthreads();
  const int nblk = st.n_blocks;
  if (warp < kDecConsumers) {
    const int grp = a.grp;
    const float* qbase = reinterpret_cast<const float*>(a.q) + (static_cast<int64_t>(s) * a.hq + h * grp) * kHeadDim;
    float qv[kMaxGroup][4], ov[kMaxGroup][4], m[kMaxGroup], l[kMaxGroup];
#pragma unroll
    for (int j = 0; j < kMaxGroup; ++j) {
      m[j] = -INFINITY;
      l[j] = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        qv[j][i] = j < grp ? qbase[j * kHeadDim + 4 * lane + i] : 0.f;
        ov[j][i] = 0.f;
      }
    }
    for (int bi = 0; bi < nblk; ++bi) {
      const int32_t blk = a.idx ? st.blocks[bi] : st.dense_lo + bi;
      const int64_t row0 = kv.block_row(s, h, blk, a.status, kIdDecode);
      if (row0 < 0) continue;
      for (int t = 16 * warp; t < 16 * warp + 16; ++t) {
        const int64_t tok = static_cast<int64_t>(blk) * kBlock + t;
        if (tok >= len) break;
        const float4 kk = *reinterpret_cast<const float4*>(k + (row0 + t) * kHeadDim + 4 * lane);
        const float4 vv = *reinterpret_cast<const float4*>(v + (row0 + t) * kHeadDim + 4 * lane);
#pragma unroll
        for (int j = 0; j < kMaxGroup; ++j) {
          if (j >= grp) break;
          float part = qv[j][0] * kk.x + qv[j][1] * kk.y + qv[j][2] * kk.z + qv[j][3] * kk.w;
#pragma unroll
          for (int off = 16; off > 0; off >>= 1) part += __shfl_xor_sync(0xffffffffu, part, off);
          const float z = part * a.scale_log2;
          const float mn = fmaxf(m[j], z);
          const float al = exp2f(m[j] - mn);
          const float p = exp2f(z - mn);
          l[j] = l[j] * al + p;
          m[j] = mn;
          ov[j][0] = ov[j][0] * al + p * vv.x;
          ov[j][1] = ov[j][1] * al + p * vv.y;
          ov[j][2] = ov[j][2] * al + p * vv.z;
          ov[j][3] = ov[j][3] * al + p * vv.w;
        }
      }
    }
    float* ob = obuf + warp * kMaxGroup * kOStride;
#pragma unroll
    for (int j = 0; j < kMaxGroup; ++j) {
      if (lane == 0) {
        st.wm[warp][j] = l[j] != l[j] ? 0.f : m[j];  // as above
        st.wl[warp][j] = l[j];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) ob[j * kOStride + 4 * lane + i] = ov[j][i];
    }
  }
  __syncthreads();
  decode_tail<float, kDecConsumers>(a, st, obuf, merge_scratch, s, h, split);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
constexpr int kDecStages = 3;

size_t decode_smem_bytes() { return 1024 + kDecStages * kStageBytes + sizeof(DecodeSmemTail); }

cudaError_t set_decode_smem() {
  cudaError_t e = cudaFuncSetAttribute(decode_bf16_kernel<kDecStages>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(decode_smem_bytes()));
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(decode_bf16_kernel<kDecStages>, cudaFuncAttributePreferredSharedMemoryCarveout,
                           cudaSharedmemCarveoutMaxShared);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(decode_bf16_kernel<kDecStages>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(decode_f32_kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                              cudaSharedmemCarveoutMaxShared);
}

// Split heuristic: fill the resident CTA slots (two 3-stage CTAs per SM) in a
// single wave: units x splits <= 2 x SMs where possible, at most
// kMaxListPerCta list entries per CTA. The bf16 kernel combines its splits in
// a thread-block cluster, so there the split count is a power of two <= 16;
// the fp32 kernel combines through global memory (up to kMaxSplits).
void decode_splits(int64_t units, int64_t list_len, int num_sms, bool cluster, bool dense, int* n_splits, int* bps) {
  const int64_t slots = 2LL * num_sms;
  int64_t want = units >= slots ? 1 : slots / units;
  if (want < 1) want = 1;
  if (cluster) {
    int64_t p = 1;
    while (p * 2 <= want && p * 2 <= 16) p *= 2;
    while (p < 16 && (list_len + p - 1) / p > kMaxListPerCta) p *= 2;
    *n_splits = static_cast<int>(p);
    *bps = static_cast<int>((list_len + p - 1) / p);
    if (*bps < 1) *bps = 1;
    return;
  }
  int64_t b = (list_len + want - 1) / want;
  if (b < 1) b = 1;
  if (!dense && b > kMaxListPerCta) b = kMaxListPerCta;
  int64_t ns = (list_len + b - 1) / b;
  if (ns > kMaxSplits) {
    b = (list_len + kMaxSplits - 1) / kMaxSplits;
    ns = (list_len + b - 1) / b;
  }
  *bps = static_cast<int>(b);
  *n_splits = static_cast<int>(ns < 1 ? 1 : ns);
}

size_t decode_partials_bytes(int64_t units, int n_splits) {
  return static_cast<size_t>(units) * n_splits * kPartFloats * sizeof(float);
}

cudaError_t launch_decode_bf16(const CUtensorMap& tmk, const CUtensorMap& tmv, const KvView& kv, int batch,
                               const DecodeArgs& a, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.n_splits, kv.hkv, batch);
  cfg.blockDim = dim3(kDecThreads, 1, 1);
  cfg.dynamicSmemBytes = decode_smem_bytes();
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = a.n_splits;  // the unit's splits form one cluster
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, decode_bf16_kernel<kDecStages>, tmk, tmv, kv, a);
}

cudaError_t launch_decode_f32(const float* k, const float* v, const KvView& kv, int batch, const DecodeArgs& a,
                              cudaStream_t stream) {
  dim3 grid(a.n_splits, kv.hkv, batch);
  decode_f32_kernel<<<grid, kDecThreads, 0, stream>>>(k, v, kv, a);
  return cudaGetLastError();
}

}  // namespace msa
