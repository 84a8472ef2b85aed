// Step 2, decode, over an e4m3 cache: softmax attention of the G query heads of
// a GQA group over the listed (or all) blocks (the arithmetic: e4m3.cuh).
//
// Bound by HBM: 2 x (128 + 4) bytes a token and KV head, 16 FLOP a byte at G = 8.
// A CTA streams its blocks through a ring of stages (a K tile and a V tile of 64 x
// 128 bytes by TMA, 128-byte swizzle, and their 64 scales each by bulk copies), two
// CTAs an SM. Eight consumer warps in two groups that take alternate blocks,
// warp w of a group tokens [16w, 16w + 16): the chain of a block (scores, exp2,
// weights, output) is longer than its share of the copy rate, so two blocks are
// worked on at a time. Two kernels: clusters of CTAs a unit where there is little
// to do, a stream over all units' blocks where there is much (see each). 1 x 1M
// tokens, 8 KV heads: 328 us, 6.75 TB/s; 8 x 128K, 32 listed blocks a head: 13.4 us.
// Measured and dropped: giving a stage back as soon as its words are in registers
// (the loads then precede the products instead of mixing with them: 634 -> 862 us
// in clusters); five stages (a stage would change groups, see kE8StreamStages).
#include "e4m3.cuh"

namespace msa {

namespace {

constexpr int kE8Threads = 32 * (kE8Consumers + 1);
constexpr int kE8Stages = 6;
constexpr int kE8StreamStages = 4;  // two CTAs an SM beside the merge buffer
// A stage belongs to one group for good (block i: group i mod 2): a group that waited
// for every other use of a stage could take an older phase of its barrier for the
// one it wants.
static_assert(kE8Stages % 2 == 0 && kE8StreamStages % 2 == 0, "stages are dealt to two groups");
constexpr int kE8MinRun = 4;
struct E8Smem {
  uint64_t full[kE8Stages];
  uint64_t empty[kE8Stages];
  int32_t valid[kE8Stages];  // of the block in the stage
  E8Next next;
  float wm[kE8Consumers][kMaxGroup];
  float wl[kE8Consumers][kMaxGroup];
  alignas(16) float xch[kPartFloats];  // the CTA's merged state (moved 16 bytes at a time)
};
constexpr size_t kE8Bytes = 1024 + static_cast<size_t>(kE8Stages) * kE8StageBytes + sizeof(E8Smem);

__device__ inline const __nv_bfloat16* e8_queries(const DecodeArgs& a, int s, int h) {
  return static_cast<const __nv_bfloat16*>(a.q) + (static_cast<int64_t>(s) * a.hq + h * a.grp) * kHeadDim;
}

// Dims 4 lane .. 4 lane + 3 of one head: O / l and the log-sum-exp.
__device__ inline void e8_write(const DecodeArgs& a, int s, int h, int head, int lane, float M, float L, float4 acc) {
  const float inv = L > 0.f ? 1.f / L : 0.f;
  const int64_t qrow = static_cast<int64_t>(s) * a.hq + h * a.grp + head;
  *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + qrow * kHeadDim + 4 * lane) =
      make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
  if (a.lse != nullptr && lane == 0) a.lse[qrow] = lse_of(M, L);
}
// One head of a state of kPartFloats.
__device__ inline void e8_store(float* part, int head, int lane, float M, float L, float4 acc) {
  if (lane == 0) {
    part[head] = M;
    part[kMaxGroup + head] = L;
  }
  *reinterpret_cast<float4*>(part + 2 * kMaxGroup + head * kHeadDim + 4 * lane) = acc;
}


// Few blocks a CTA: one cluster of n_splits CTAs a unit, joined through
// distributed shared memory. grid (n_splits, Hkv, batch)
__global__ void __launch_bounds__(kE8Threads, 2)
    decode_e4m3_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                       const float* __restrict__ k_scale, const float* __restrict__ v_scale, KvView kv, DecodeArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* ring = smem_align1024(smem_raw);
  uint8_t* scales = ring + kE8Stages * 2 * kE8Tile;  // [stage][K 64 | V 64] floats
  E8Smem& sh = *reinterpret_cast<E8Smem*>(scales + kE8Stages * 2 * kE8ScaleBytes);

  const int split = blockIdx.x, h = blockIdx.y, s = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kE8Stages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], kE8Group);
    }
    fence_mbar_init();
  }
  if (warp == kE8Consumers && lane == 0) {
    tma_prefetch_desc(&tmk);
    tma_prefetch_desc(&tmv);
  }
  pdl_wait();  // the index lists (and every other input) come from earlier work
  int lo, nblk;  // list entries, or an equal share of this sequence's own blocks
  int32_t first = -1;  // the producer lane's first entry, on its way while the length is
  const int32_t* list = nullptr;
  if (a.idx != nullptr) {
    lo = min(a.k_total, split * a.bps);
    nblk = min(a.k_total, lo + a.bps) - lo;
    list = a.idx + (static_cast<int64_t>(s) * a.hkv + h) * a.k_total + lo;
    if (warp == kE8Consumers && lane < nblk) first = list[lane];
  }
  const int64_t len = kv.seq_len(s, a.status, kIdDecode);
  if (a.idx == nullptr) {
    const int64_t nb = (len + kBlock - 1) / kBlock;
    lo = static_cast<int>(nb * split / a.n_splits);
    nblk = static_cast<int>(nb * (split + 1) / a.n_splits) - lo;
  }
  __syncthreads();
  E8Consumer w;
  if (warp == kE8Consumers) {
    e8_produce<kE8Stages>(&tmk, &tmv, k_scale, v_scale, nblk, ring, scales, sh.full, sh.empty, sh.valid, sh.next,
                          a.status, lane, [&](int i, int64_t& row, int32_t& valid) {
                            e8_find(kv, s, h, list == nullptr ? lo + i : i < 32 ? first : list[i], len, a.status, row,
                                    valid);
                          });
  } else {
    w.start(e8_queries(a, s, h), a.grp, a.scale_log2, lane);
    const int w16 = 16 * (warp & 3);
    for (int i = warp >> 2; i < nblk; i += 2) {
      const int stg = i % kE8Stages;
      if (!mbar_wait_warp(&sh.full[stg], (i / kE8Stages) & 1, a.status, kIdDecode)) break;
      const int valid = sh.valid[stg];
      if (w16 < valid)
        w.block(smem_u32(ring + stg * 2 * kE8Tile),
                reinterpret_cast<const float*>(scales + stg * 2 * kE8ScaleBytes), valid, w16, lane);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.empty[stg]);
    }
    w.finish();
  }
  pdl_trigger();  // the next kernel may start its set-up
  if (warp < kE8Consumers) {
    bar_sync_warps(1, 32 * kE8Consumers);  // every consumer is done with the ring: reuse it for the merge
    float M, L;
    float4 acc;
    w.merge(reinterpret_cast<float*>(ring), sh.wm, sh.wl, warp, lane, [] {}, M, L, acc);
    if (a.n_splits > 1) e8_store(sh.xch, warp, lane, M, L, acc);
    else if (warp < a.grp) e8_write(a, s, h, warp, lane, M, L, acc);
  }
  if (a.n_splits > 1) cluster_join<__nv_bfloat16>(a, sh.xch, s, h);
}

__device__ inline int e8_blocks(int tokens) { return tokens / kBlock + (tokens % kBlock != 0 ? 1 : 0); }

// The unit under way in a walk over the positions.
struct E8Unit {
  int s, h;
  int start, len, tokens;  // positions [start, start + len); tokens of the sequence
  __device__ void load(const KvView& kv, const DecodeArgs& a) {
    tokens = static_cast<int>(kv.seq_len(s, a.status, kIdDecode));
    len = a.idx != nullptr ? a.k_total : e8_blocks(tokens);
  }
  __device__ void next(const KvView& kv, const DecodeArgs& a) {  // only where a later unit has positions
    start += len;
    if (++h < a.hkv) return;
    h = 0;
    do {
      ++s;
      load(kv, a);
    } while (len == 0);
  }
};

// Many blocks a CTA: the blocks (list entries) of all units laid end to end, unit
// after unit, and dealt in equal runs to the CTAs of one wave, whatever the
// lengths of the sequences. A CTA streams its run without a break; where a unit
// ends in it, the warps' states are merged: into the output if the whole unit was
// its own, else into a partial of the workspace (slot 0: the unit the run begins
// in, slot 1: the one it ends in), and the last of the unit's CTAs to arrive, by a
// ticket that nobody waits for, joins the partials.
struct E8Stream {
  uint64_t full[kE8StreamStages];
  uint64_t empty[kE8StreamStages];
  int32_t sums[kE8Threads / 32];
  int32_t s0, at0;  // the sequence of the first unit, the position at which it begins
  int32_t lo, hi;   // this CTA's run
  E8Unit unit[kE8Consumers];  // each consumer warp's place in it: kept here, for the block loop needs the registers
  E8Unit join[2];  // units this CTA holds a part of (slots 0, 1) ...
  int32_t arrived[2];  // ... and how many CTAs had arrived with it (0: no such unit)
  int32_t valid[kE8StreamStages];
  E8Next next;
  float wm[2][kE8Consumers][kMaxGroup];  // of alternate merges
  float wl[2][kE8Consumers][kMaxGroup];
};
constexpr size_t kE8StreamBytes =
    1024 + static_cast<size_t>(kE8StreamStages) * kE8StageBytes + 2 * kE8MergeBytes + sizeof(E8Stream);

// CTAs with a run: kE8MinRun positions or more each, as long as there are that many.
__device__ inline int e8_runs(int T) {
  return min(static_cast<int>(gridDim.x), T / kE8MinRun + (T % kE8MinRun != 0 ? 1 : 0));  // T may be 2^31 - 2
}
// Positions [0, T) dealt to n <= T CTAs: the first T % n get one more.
struct E8Deal {
  int n, base, more;
  __device__ E8Deal(int T, int n_) : n(n_), base(T / n_), more(T - T / n_ * n_) {}
  __device__ int first(int cta) const { return cta * base + min(cta, more); }
  __device__ int cta_of(int x) const {
    const int b = more * (base + 1);
    return x < b ? x / (base + 1) : more + (x - b) / base;
  }
};

__global__ void __launch_bounds__(kE8Threads, 2)
    decode_e4m3_stream_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                              const float* __restrict__ k_scale, const float* __restrict__ v_scale, KvView kv,
                              DecodeArgs a, int batch) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* ring = smem_align1024(smem_raw);
  uint8_t* scales = ring + kE8StreamStages * 2 * kE8Tile;
  float* merge = reinterpret_cast<float*>(scales + kE8StreamStages * 2 * kE8ScaleBytes);
  E8Stream& st = *reinterpret_cast<E8Stream*>(reinterpret_cast<uint8_t*>(merge) + 2 * kE8MergeBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kE8StreamStages; ++i) {
      mbar_init(&st.full[i], 1);
      mbar_init(&st.empty[i], kE8Group);
    }
    fence_mbar_init();
    st.arrived[0] = st.arrived[1] = 0;
  }
  if (warp == kE8Consumers && lane == 0) {
    tma_prefetch_desc(&tmk);
    tma_prefetch_desc(&tmv);
  }
  pdl_wait();  // the index lists (and every other input) come from earlier work

  // Positions of all units: T, this CTA's [lo, hi) of them and the unit at lo.
  E8Unit u;
  int T = 0, s0 = 0, at0 = 0;  // at0: the position at which sequence s0 begins
  E8Deal deal(1, 1);
  int lo = 0;
  if (batch <= 32) {  // every warp by itself
    u.s = min(lane, batch - 1);
    u.load(kv, a);
    const int own = lane < batch ? u.len * a.hkv : 0;
    int incl = own;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += v;
    }
    T = __shfl_sync(0xffffffffu, incl, 31);
    deal = E8Deal(T, max(1, e8_runs(T)));
    lo = deal.first(blockIdx.x);
    s0 = __ffs(__ballot_sync(0xffffffffu, lo >= incl - own && lo < incl)) - 1;  // -1: no run
    at0 = __shfl_sync(0xffffffffu, incl - own, max(s0, 0));
    __syncthreads();
  } else {
    const int per = (batch + kE8Threads - 1) / kE8Threads;
    const int sa = min(batch, tid * per), sb = min(batch, sa + per);
    int own = 0;
    for (u.s = sa; u.s < sb; ++u.s) {
      u.load(kv, a);
      own += u.len * a.hkv;
    }
    int incl = own;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += v;
    }
    if (lane == 31) st.sums[warp] = incl;
    __syncthreads();
    int excl = incl - own;
    for (int i = 0; i < kE8Threads / 32; ++i) {
      if (i < warp) excl += st.sums[i];
      T += st.sums[i];
    }
    deal = E8Deal(T, max(1, e8_runs(T)));
    lo = deal.first(blockIdx.x);
    if (lo >= excl && lo < excl + own) {
      u.s = sa;
      u.load(kv, a);
      while (lo >= excl + u.len * a.hkv) {
        excl += u.len * a.hkv;
        ++u.s;
        u.load(kv, a);
      }
      st.s0 = u.s;
      st.at0 = excl;
    }
    __syncthreads();
    s0 = st.s0;
    at0 = st.at0;
  }
  // sequences without a block: nobody's run holds them
  for (int s = blockIdx.x; s < batch; s += gridDim.x) {
    u.s = s;
    u.load(kv, a);
    if (u.len != 0) continue;
    for (int i = tid; i < a.hq * 16; i += kE8Threads)
      reinterpret_cast<uint4*>(a.out)[static_cast<int64_t>(s) * a.hq * 16 + i] = make_uint4(0u, 0u, 0u, 0u);
    if (a.lse != nullptr)
      for (int i = tid; i < a.hq; i += kE8Threads) a.lse[static_cast<int64_t>(s) * a.hq + i] = -INFINITY;
  }
  if (static_cast<int>(blockIdx.x) >= e8_runs(T)) return;
  const int hi = deal.first(blockIdx.x + 1);
  u.s = s0;
  u.load(kv, a);
  u.h = (lo - at0) / u.len;
  u.start = at0 + u.h * u.len;

  if (warp == kE8Consumers) {
    e8_produce<kE8StreamStages>(&tmk, &tmv, k_scale, v_scale, hi - lo, ring, scales, st.full, st.empty, st.valid, st.next,
                                a.status, lane, [&](int i, int64_t& row, int32_t& valid) {
                                  const int x = lo + i;
                                  while (x >= u.start + u.len) u.next(kv, a);
                                  int64_t blk = x - u.start;
                                  if (a.idx != nullptr)
                                    blk = a.idx[(static_cast<int64_t>(u.s) * a.hkv + u.h) * a.k_total + blk];
                                  e8_find(kv, u.s, u.h, blk, u.tokens, a.status, row, valid);
                                });
    return;
  }

  // ---------------- consumers ----------------
  constexpr int kConsumerThreads = 32 * kE8Consumers;
  E8Consumer w;
  w.start(e8_queries(a, u.s, u.h), a.grp, a.scale_log2, lane);
  E8Unit& at = st.unit[warp];
  if (lane == 0) at = u;
  if (tid == 0) {
    st.lo = lo;
    st.hi = hi;
  }
  bar_sync_warps(1, kConsumerThreads);
  bool alive = true;
  int odd = 0;
  for (int x = lo; x < st.hi;) {
    const int i1 = min(st.hi, at.start + at.len) - st.lo;
    int i = x - st.lo;
    i += (i ^ (warp >> 2)) & 1;  // the groups take alternate blocks of the run
    for (; alive && i < i1; i += 2) {
      const int stg = i % kE8StreamStages;
      alive = mbar_wait_warp(&st.full[stg], (i / kE8StreamStages) & 1, a.status, kIdDecode);
      if (!alive) break;
      const int valid = st.valid[stg], w16 = 16 * (warp & 3);
      if (w16 < valid)
        w.block(smem_u32(ring + stg * 2 * kE8Tile),
                reinterpret_cast<const float*>(scales + stg * 2 * kE8ScaleBytes), valid, w16, lane);
      __syncwarp();
      if (lane == 0) mbar_arrive(&st.empty[stg]);
    }
    w.finish();
    const E8Unit done = at;
    const int end = i1 + st.lo;
    float M, L;
    float4 acc;
    w.merge(merge + odd * (kE8MergeBytes / sizeof(float)), st.wm[odd], st.wl[odd], warp, lane,
            [&] {  // the second group loads the next unit's queries while the first joins the states
              if (end >= st.hi) return;
              E8Unit next = done;
              next.next(kv, a);
              w.start(e8_queries(a, next.s, next.h), a.grp, a.scale_log2, lane);
              __syncwarp();
              if (lane == 0) at = next;
              __syncwarp();
            },
            M, L, acc);
    if (x == done.start && end == done.start + done.len) {
      if (warp < a.grp) e8_write(a, done.s, done.h, warp, lane, M, L, acc);
    } else {  // announced at the end of the run: nothing here waits for memory
      const int k = x == st.lo ? 0 : 1;
      e8_store(a.partials + (2 * static_cast<int64_t>(blockIdx.x) + k) * kPartFloats, warp, lane, M, L, acc);
      if (tid == 0) {
        st.join[k] = done;
        st.arrived[k] = -1;
      }
    }
    odd ^= 1;
    x = end;
  }
  pdl_trigger();  // the next kernel may start its set-up
  bar_sync_warps(1, kConsumerThreads);
  if (tid < 2 && st.arrived[tid] != 0) {
    __threadfence();
    st.arrived[tid] = 1 + atomicAdd(&a.tickets[static_cast<int64_t>(st.join[tid].s) * a.hkv + st.join[tid].h], 1);
  }
  bar_sync_warps(1, kConsumerThreads);
  for (int k = 0; k < 2; ++k) {
    if (st.arrived[k] == 0) continue;
    const E8Unit j = st.join[k];
    const int c0 = deal.cta_of(j.start), parts = deal.cta_of(j.start + j.len - 1) - c0 + 1;  // its CTAs
    if (st.arrived[k] != parts) continue;  // a later CTA joins the unit
    __threadfence();
    if (tid == 0) a.tickets[static_cast<int64_t>(j.s) * a.hkv + j.h] = 0;  // ready for the next call
    const int late = j.start != deal.first(c0) ? 1 : 0;  // the first CTA's partial is in its slot 1
    const float* base = a.partials + 2 * static_cast<int64_t>(c0) * kPartFloats;
    auto part_of = [&](int p) { return base + (2 * p + (p == 0 ? late : 0)) * kPartFloats; };
    // warp w: head w. Its factors 2^(m - M), 32 partials at a time in a register a lane.
    if (warp >= a.grp) continue;
    float Mx = -INFINITY, Lx = 0.f;
    float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
    const int ofs = 2 * kMaxGroup + warp * kHeadDim + 4 * lane;  // dims 4 lane .. 4 lane + 3
    for (int p0 = 0; p0 < parts; p0 += 32) {
      const int p = p0 + lane, m = min(32, parts - p0);
      const float pm = p < parts ? __ldcg(part_of(p) + warp) : -INFINITY;
      const float pl = p < parts ? __ldcg(part_of(p) + kMaxGroup + warp) : 0.f;
      float top = pm;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
      top = fmaxf(top, Mx);
      const float ref = top == -INFINITY ? 0.f : top;
      const float f = exp2f(pm - ref), fx = exp2f(Mx - ref);
      float sum = f * pl;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      Lx = Lx * fx + sum;
      r.x *= fx; r.y *= fx; r.z *= fx; r.w *= fx;
      Mx = top;
      for (int i0 = 0; i0 < m; i0 += 8) {  // eight partials in flight
        float4 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          v[i] = i0 + i < m ? __ldcg(reinterpret_cast<const float4*>(part_of(p0 + i0 + i) + ofs))
                            : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float fi = __shfl_sync(0xffffffffu, f, i0 + i);  // 0 past the last
          r.x = fmaf(fi, v[i].x, r.x); r.y = fmaf(fi, v[i].y, r.y);
          r.z = fmaf(fi, v[i].z, r.z); r.w = fmaf(fi, v[i].w, r.w);
        }
      }
    }
    e8_write(a, j.s, j.h, warp, lane, Mx, Lx, r);
  }
}

}  // namespace

// Clusters of `c` CTAs that the device holds at once (0 on an error).
int decode_e4m3_max_clusters(int c) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(c, 1, 1);
  cfg.blockDim = dim3(kE8Threads, 1, 1);
  cfg.dynamicSmemBytes = kE8Bytes;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = c;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, decode_e4m3_kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return n;
}

size_t decode_e4m3_partials_bytes(int num_sms) {
  return static_cast<size_t>(2 * num_sms) * 2 * kPartFloats * sizeof(float);
}

// Which kernel and how wide: returns the stream's CTAs (one wave of two an SM),
// or 0 for clusters of *n_splits CTAs with *bps list entries each. Costs in
// microseconds as measured: a block takes a CTA 0.79 when all 2 num_sms of
// them stream (its share of the copy rate), less in proportion when fewer do, but
// 0.60 at least; a cluster CTA has set-up, first loads and the join worth 6
// blocks, a stream CTA (two prefix sums, up to two joins in memory) 20, and 5 for
// every unit that ends in it. Clusters take the power of two whose waves cost
// least. Measured
// (clusters / stream, us): 64 units of 32 blocks 12 / 19, 256 of 32 27 / 35, 8
// of 1050 59 / 39, 8 of 16384 637 / 328. Where every block is attended and the
// batch has several sequences, the host knows their longest possible length
// alone: a cluster's time is set by it, the stream's by what is there, taken as
// 0.6 of it (48 units of up to 512 blocks, lengths log-uniform over a factor of 32:
// 63 / 31; all at the full length, 256 units of 128 blocks: 89 / 95).
int decode_e4m3_shape(int64_t units, int64_t list_len, bool ragged, int num_sms, const int* max_clusters,
                      int* n_splits, int* bps) {
  const double slots = 2.0 * num_sms;
  double best = -1;
  for (int i = 0; i < 5; ++i) {
    const int64_t p = int64_t(1) << i;
    if (i > 0 && (max_clusters[i] < 1 || list_len < p)) break;
    const int64_t at_once = max_clusters[i] > 0 ? max_clusters[i] : 1;
    const int64_t waves = (units + at_once - 1) / at_once, each = (list_len + p - 1) / p;
    const double used = static_cast<double>(units * p) / (waves * slots);
    const double cost = static_cast<double>(waves * (each + 6)) * (0.79 * used > 0.60 ? 0.79 * used : 0.60);
    if (best < 0 || cost < best) {
      best = cost;
      *n_splits = static_cast<int>(p);
      *bps = static_cast<int>(each < 1 ? 1 : each);
    }
  }
  if (units * list_len >= INT32_MAX) return 0;  // the stream counts positions in 32 bits
  const double blocks = static_cast<double>(units) * ((ragged ? 0.6 : 1.0) * static_cast<double>(list_len) + 5);
  return (blocks / slots + 20) * 0.79 < best ? 2 * num_sms : 0;
}

cudaError_t set_decode_e4m3_smem() {
  cudaError_t e0 = cudaFuncSetAttribute(decode_e4m3_stream_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        static_cast<int>(kE8StreamBytes));
  if (e0 != cudaSuccess) return e0;
  e0 = cudaFuncSetAttribute(decode_e4m3_stream_kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                            cudaSharedmemCarveoutMaxShared);
  if (e0 != cudaSuccess) return e0;
  cudaError_t e = cudaFuncSetAttribute(decode_e4m3_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(kE8Bytes));
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(decode_e4m3_kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                           cudaSharedmemCarveoutMaxShared);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(decode_e4m3_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
}

cudaError_t launch_decode_e4m3(const CUtensorMap& tmk, const CUtensorMap& tmv, const float* k_scale,
                               const float* v_scale, const KvView& kv, int batch, const DecodeArgs& a,
                               int stream_ctas, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kE8Threads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  if (stream_ctas > 0) {
    cfg.gridDim = dim3(stream_ctas, 1, 1);
    cfg.dynamicSmemBytes = kE8StreamBytes;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, decode_e4m3_stream_kernel, tmk, tmv, k_scale, v_scale, kv, a, batch);
  }
  cfg.gridDim = dim3(a.n_splits, kv.hkv, batch);
  cfg.dynamicSmemBytes = kE8Bytes;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = a.n_splits;  // the unit's splits form one cluster
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, decode_e4m3_kernel, tmk, tmv, k_scale, v_scale, kv, a);
}

}  // namespace msa
