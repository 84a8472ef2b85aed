// Where the tokens of a step go: sequences grow (pages popped off a stack of
// free pages, positions and cache slots of the new tokens) and shrink (pages
// pushed back), on the GPU, from lengths and counts in its memory: a step of single tokens never
// takes them to the host (a batch of prefill chunks does: those calls take starts and counts there).
//
// With n_s the length of sequence s, c_s its new tokens and B = 64 tokens a
// block:
//   have_s = ceil(n_s / B),  need_s = ceil((n_s + c_s) / B) - have_s
//   O_s = sum_{u < s} c_u,   P_s = sum_{u < s} need_u      (prefix sums)
//   new block have_s + i of s gets page free[F - 1 - (P_s + i)]
//   token r of s is row O_s + r: position n_s + r, slot page * B + offset.
//
// What bounds it: one launch. A step reads and writes a few KB to a few MB, so
// nothing may be exchanged between CTAs on the critical path: every CTA
// computes both prefix sums over the whole batch itself (at most
// kMaxSeqBatch sequences, 8 bytes each, from L2) into shared memory and then
// takes its stripe of the rows, each row finding its sequence by a binary
// search there. The one exchange is a ticket that nobody waits for: the last
// CTA to finish writes the new lengths and the new stack height, so that both
// may replace the arrays that the other CTAs read. 1 token 2.9 us, 131072 rows of 32
// ragged chunks 5.1 us, trimming 32 sequences of up to 1M tokens 4.0 us (an empty
// kernel between two others: about 2). 256 threads and a row a thread: 512 threads
// and four rows took 3.2, 6.6 and 4.7.
#include "kernels.cuh"

namespace msa {

namespace {

constexpr int kSeqThreads = 256;

// Exclusive prefix sums of (a, b) over the CTA's threads, and their totals.
__device__ inline void block_scan2(int64_t& a, int64_t& b, int64_t& ta, int64_t& tb) {
  __shared__ int64_t wa[kSeqThreads / 32], wb[kSeqThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t ia = a, ib = b;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t ua = __shfl_up_sync(0xffffffffu, ia, off), ub = __shfl_up_sync(0xffffffffu, ib, off);
    if (lane >= off) {
      ia += ua;
      ib += ub;
    }
  }
  if (lane == 31) {
    wa[warp] = ia;
    wb[warp] = ib;
  }
  __syncthreads();
  int64_t ba = 0, bb = 0;
  ta = tb = 0;
#pragma unroll
  for (int w = 0; w < kSeqThreads / 32; ++w) {
    if (w == warp) {
      ba = ta;
      bb = tb;
    }
    ta += wa[w];
    tb += wb[w];
  }
  a = ba + ia - a;
  b = bb + ib - b;
}

// The sequence whose rows [off[s], off[s + 1]) hold row j < off[n].
__device__ inline int seq_of_row(const int32_t* off, int n, int32_t j) {
  int lo = 0, hi = n;  // off[lo] <= j < off[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= j) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ inline int64_t blocks_of(int64_t tokens) { return (tokens + kBlock - 1) / kBlock; }

// True in every thread of the CTA that finishes last (grid of several CTAs:
// one ticket, reset by that CTA; a single CTA needs none). Every read that the
// CTA made of the arrays about to be replaced comes before it.
__device__ inline bool last_cta(int32_t* ticket) {
  __shared__ int last;
  if (gridDim.x == 1) {
    __syncthreads();
    return true;
  }
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    last = atomicAdd(ticket, 1) == static_cast<int>(gridDim.x) - 1;
    if (last) *ticket = 0;  // ready for the next call
  }
  __syncthreads();
  return last != 0;
}

__global__ void __launch_bounds__(kSeqThreads) extend_sequences_kernel(KvView kv, ExtendArgs a) {
  extern __shared__ int32_t sm[];
  pdl_wait();
  pdl_trigger();
  int32_t* q_off = sm;              // [batch + 1] first row of each sequence
  int32_t* p_off = sm + a.batch + 1;  // [batch + 1] first new page of each sequence
  const bool paged = kv.layout == MSA_KV_PAGED;
  const int64_t cap = min(kv.capacity(), static_cast<int64_t>(INT32_MAX));
  const int per = (a.batch + kSeqThreads - 1) / kSeqThreads;
  const int s0 = min(a.batch, static_cast<int>(threadIdx.x) * per), s1 = min(a.batch, s0 + per);
  int bad = 0;
  int64_t tok = 0, pg = 0;
  for (int s = s0; s < s1; ++s) {
    const int64_t n = kv.seq_lens[s], c = a.q_counts[s];
    bad |= n < 0 || c < 0 || n + c > cap;
    tok += c;
    pg += blocks_of(n + c) - blocks_of(n);
  }
  int64_t T = 0, P = 0;
  block_scan2(tok, pg, T, P);
  bad = __syncthreads_or(bad);
  const int64_t F = paged ? *a.free_count : 0;
  int code = bad ? MSA_ERR_DEVICE_BOUNDS : MSA_OK;
  if (T > a.n_slots || (paged && (F < 0 || F > kv.num_pages))) code = MSA_ERR_DEVICE_BOUNDS;
  if (code == MSA_OK && paged && P > F) code = MSA_ERR_OUT_OF_PAGES;
  if (code != MSA_OK) {  // all or nothing
    T = P = 0;
    if (blockIdx.x == 0 && threadIdx.x == 0) set_status(a.status, code, kIdExtend);
  }
  for (int s = s0; s < s1; ++s) {
    q_off[s] = code == MSA_OK ? static_cast<int32_t>(tok) : 0;
    p_off[s] = code == MSA_OK ? static_cast<int32_t>(pg) : 0;
    const int64_t n = kv.seq_lens[s], c = a.q_counts[s];
    tok += c;
    pg += blocks_of(n + c) - blocks_of(n);
  }
  if (threadIdx.x == 0) q_off[a.batch] = static_cast<int32_t>(T);
  __syncthreads();

  const int64_t stride = static_cast<int64_t>(gridDim.x) * kSeqThreads;
  for (int64_t j = static_cast<int64_t>(blockIdx.x) * kSeqThreads + threadIdx.x; j < a.n_slots; j += stride) {
    int32_t pos = 0;
    int64_t slot = -1;
    if (j < T) {
      const int s = seq_of_row(q_off, a.batch, static_cast<int32_t>(j));
      const int32_t n = kv.seq_lens[s];
      pos = n + (static_cast<int32_t>(j) - q_off[s]);
      if (!paged) {
        slot = s * kv.max_tokens + pos;
      } else {
        const int64_t b = pos / kBlock, fresh = b - blocks_of(n);
        int32_t* entry = a.page_table + static_cast<int64_t>(s) * kv.max_pages + b;
        int32_t page = fresh >= 0 ? a.free_pages[F - 1 - (p_off[s] + fresh)]
                                  : kv.page_table[static_cast<int64_t>(s) * kv.max_pages + b];
        if (page < 0 || page >= kv.num_pages) {
          set_status(a.status, MSA_ERR_DEVICE_BOUNDS, kIdExtend);
          page = -1;
        } else {
          slot = static_cast<int64_t>(page) * kBlock + pos % kBlock;
        }
        if (fresh >= 0 && pos % kBlock == 0) *entry = page;  // every new block begins with one of the rows
      }
    }
    a.positions[j] = pos;
    a.slots[j] = slot;
  }
  if (blockIdx.x == 0)
    for (int s = threadIdx.x; s <= a.batch; s += kSeqThreads) a.q_off[s] = q_off[s];
  if (!last_cta(a.ticket)) return;
  for (int s = threadIdx.x; s < a.batch; s += kSeqThreads) {
    const int32_t n = kv.seq_lens[s], c = code == MSA_OK ? a.q_counts[s] : 0;
    a.seq_lens_out[s] = n + c;
  }
  if (paged && threadIdx.x == 0) *a.free_count_out = static_cast<int32_t>(F - P);
}

__global__ void __launch_bounds__(kSeqThreads) trim_sequences_kernel(KvView kv, TrimArgs a) {
  extern __shared__ int32_t sm[];
  pdl_wait();
  pdl_trigger();
  int32_t* off = sm;  // [batch + 1] first freed page of each sequence
  const bool paged = kv.layout == MSA_KV_PAGED;
  const int64_t cap = min(kv.capacity(), static_cast<int64_t>(INT32_MAX));
  const int per = (a.batch + kSeqThreads - 1) / kSeqThreads;
  const int s0 = min(a.batch, static_cast<int>(threadIdx.x) * per), s1 = min(a.batch, s0 + per);
  int bad = 0;
  int64_t pg = 0, unused = 0;
  for (int s = s0; s < s1; ++s) {
    const int64_t n = kv.seq_lens[s], keep = a.keep_lens[s];
    bad |= n < 0 || n > cap || keep < 0;
    pg += blocks_of(n) - blocks_of(min(n, keep));
  }
  int64_t P = 0, U = 0;
  block_scan2(pg, unused, P, U);
  bad = __syncthreads_or(bad);
  const int64_t F = paged ? *a.free_count : 0;
  if (paged && !bad) bad = F < 0 || F + P > kv.num_pages;
  if (bad) {  // all or nothing
    P = 0;
    if (blockIdx.x == 0 && threadIdx.x == 0) set_status(a.status, MSA_ERR_DEVICE_BOUNDS, kIdTrim);
  }
  for (int s = s0; s < s1; ++s) {
    off[s] = bad ? 0 : static_cast<int32_t>(pg);
    const int64_t n = kv.seq_lens[s], keep = a.keep_lens[s];
    pg += blocks_of(n) - blocks_of(min(n, keep));
  }
  if (threadIdx.x == 0) off[a.batch] = static_cast<int32_t>(P);
  __syncthreads();
  if (paged) {
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kSeqThreads;
    for (int64_t j = static_cast<int64_t>(blockIdx.x) * kSeqThreads + threadIdx.x; j < P; j += stride) {
      const int s = seq_of_row(off, a.batch, static_cast<int32_t>(j));
      const int64_t kept = min(kv.seq_lens[s], a.keep_lens[s]);
      a.free_pages[F + j] = kv.page(s, blocks_of(kept) + j - off[s], a.status, kIdTrim);
    }
  }
  if (!last_cta(a.ticket)) return;
  for (int s = threadIdx.x; s < a.batch; s += kSeqThreads) {
    const int32_t n = kv.seq_lens[s];
    a.seq_lens_out[s] = bad ? n : min(n, a.keep_lens[s]);
  }
  if (paged && threadIdx.x == 0) *a.free_count_out = static_cast<int32_t>(F + P);
}

int seq_grid(int64_t rows, int num_sms) {
  int64_t g = (rows + kSeqThreads - 1) / kSeqThreads;
  if (g > 2LL * num_sms) g = 2LL * num_sms;
  return static_cast<int>(g < 1 ? 1 : g);
}

}  // namespace

cudaError_t set_sequences_smem() {
  const int bytes = 2 * (kMaxSeqBatch + 1) * static_cast<int>(sizeof(int32_t));
  cudaError_t e = cudaFuncSetAttribute(extend_sequences_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(trim_sequences_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

cudaError_t launch_extend_sequences(const KvView& kv, const ExtendArgs& a, int num_sms, cudaStream_t stream) {
  const size_t smem = 2 * (static_cast<size_t>(a.batch) + 1) * sizeof(int32_t);
  return launch_overlapped(extend_sequences_kernel, seq_grid(a.n_slots, num_sms), kSeqThreads, smem, stream, kv, a);
}

cudaError_t launch_trim_sequences(const KvView& kv, const TrimArgs& a, int num_sms, cudaStream_t stream) {
  const size_t smem = (static_cast<size_t>(a.batch) + 1) * sizeof(int32_t);
  const int64_t most = kv.layout == MSA_KV_PAGED
                           ? (static_cast<int64_t>(a.batch) * kv.max_pages < kv.num_pages
                                  ? static_cast<int64_t>(a.batch) * kv.max_pages
                                  : kv.num_pages)
                           : 1;
  return launch_overlapped(trim_sequences_kernel, seq_grid(most, num_sms), kSeqThreads, smem, stream, kv, a);
}

}  // namespace msa
