// The page plan of one serving step: how many pages each sequence gains, which ones, and where
// every new token goes.  Integer work, bound by latency for a decode step and by its 20 written
// bytes per token for a prefill.
//
// Two prefix sums over the sequences (tokens, pages) decide everything, so every CTA computes
// both for itself from the 8 bytes per sequence it reads (L2 after the first CTA) and keeps
// them in shared memory (12 bytes per sequence, 192 KB at most); no CTA waits for another and one launch does the step.  Then each
// thread finds the sequence of its two tokens by bisection in shared memory.  A new page starts
// with a new token, and that token's thread enters the page into the block table.
#include "common.cuh"

namespace csa2 {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanMaxSeqs = 16384;

struct PlanArgs {
  int num_seqs;
  const int32_t* old_len;
  const int32_t* new_len;
  int max_tokens;
  int32_t* block_table;
  int max_pages;
  const int32_t* free_pages;
  int num_free;
  const int32_t* free_used;
  int32_t* free_used_out;
  int32_t* seq_len;
  int32_t* tok_start;
  int32_t* q_seq;
  int64_t* q_pos;
  int64_t* rows;
  int* status;
};

__device__ __forceinline__ int64_t warp_inclusive(int64_t x) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
    if ((threadIdx.x & 31) >= d) x += y;
  }
  return x;
}
// exclusive prefix of v over the block's threads; *total gets the sum
__device__ __forceinline__ int64_t block_prefix(int64_t v, int64_t* warp_sum, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int64_t x = warp_inclusive(v);
  __syncthreads();                       // an earlier prefix's sums have been read
  if (lane == 31) warp_sum[warp] = x;
  __syncthreads();
  if (warp == 0) {
    const int64_t s = warp_inclusive(lane < warps ? warp_sum[lane] : 0);
    __syncwarp();
    if (lane < warps) warp_sum[lane] = s;
  }
  __syncthreads();
  *total = warp_sum[warps - 1];
  return (warp ? warp_sum[warp - 1] : 0) + x - v;
}

__global__ void __launch_bounds__(kPlanThreads) plan_pages_kernel(const PlanArgs a) {
  extern __shared__ int32_t plan_smem[];
  int32_t* tok = plan_smem;                       // [num_seqs + 1] first token
  int32_t* page0 = plan_smem + a.num_seqs + 1;    // [num_seqs] first free_pages entry; -1: refused
                                                  // (before that, the new lengths)
  int32_t* held = page0 + a.num_seqs;             // [num_seqs] stored entries
  __shared__ int64_t warp_sum[kPlanThreads / 32];
  __shared__ int granted_pages;
  pdl_trigger();
  pdl_wait();
  const bool writer = blockIdx.x == 0;            // of the per-sequence outputs
  const int tid = threadIdx.x, S = a.num_seqs;
  const int per = (S + (int)blockDim.x - 1) / (int)blockDim.x;
  const int s0 = min(S, tid * per), s1 = min(S, s0 + per);
  if (tid == 0) granted_pages = 0;

  bool negative = false;
  for (int s = tid; s < S; s += blockDim.x) {     // one coalesced read of both lengths
    const int o = __ldg(a.old_len + s), n = __ldg(a.new_len + s);
    negative |= o < 0 || n < 0;
    held[s] = max(o, 0);
    page0[s] = max(n, 0);
  }
  int used = __ldg(a.free_used);
  __syncthreads();
  int64_t sum = 0, total, pages_total;
  for (int s = s0; s < s1; ++s) sum += page0[s];
  const int64_t tok_base = block_prefix(sum, warp_sum, &total);
  const int64_t most = (int64_t)a.max_pages * kPageRows;

  // pages a sequence needs; 0 and *fits false where table or token arrays do not hold it
  auto need = [&](int s, int64_t at, bool* fits) -> int {
    const int64_t o = held[s], n = page0[s];
    *fits = o + n <= most && at + n <= a.max_tokens;
    return *fits ? (int)((o + n + kPageRows - 1) / kPageRows - (o + kPageRows - 1) / kPageRows) : 0;
  };
  int64_t at = tok_base;
  sum = 0;
  for (int s = s0; s < s1; ++s) {
    bool fits;
    sum += need(s, at, &fits);
    at += page0[s];
  }
  int64_t upto = block_prefix(sum, warp_sum, &pages_total);
  const bool bad_used = used < 0 || used > a.num_free;
  if (bad_used) used = a.num_free;
  const int avail = a.num_free - used;

  at = tok_base;
  bool refused = false;
  int taken = 0;
  for (int s = s0; s < s1; ++s) {
    bool fits;
    const int w = need(s, at, &fits);
    const bool grant = fits && (w == 0 || upto + w <= avail);
    const int o = held[s], n = page0[s];
    tok[s] = (int32_t)min(at, (int64_t)a.max_tokens);
    page0[s] = grant ? used + (int)(w == 0 ? 0 : upto) : -1;
    refused |= !grant;
    if (grant && w > 0) taken = (int)upto + w;
    if (writer) {
      a.seq_len[s] = grant ? o + n : o;
      a.tok_start[s] = tok[s];
    }
    upto += w;
    at += n;
  }
  if (taken > 0) atomicMax(&granted_pages, taken);
  if (tid == 0) tok[S] = (int32_t)min(total, (int64_t)a.max_tokens);
  __syncthreads();
  if (writer) {
    if (tid == 0) {
      a.tok_start[S] = tok[S];
      a.free_used_out[0] = used + granted_pages;
      if (bad_used) report(a.status, CSA2_ERR_INVALID_ARG);
    }
    if (negative) report(a.status, CSA2_ERR_INVALID_ARG);
    if (refused) report(a.status, CSA2_ERR_CAPACITY);
  }

  // two tokens per thread: the maps' stores are 8 and 16 bytes wide and coalesced
  const int n_tok = tok[S];
  for (int64_t t0 = ((int64_t)blockIdx.x * blockDim.x + tid) * 2; t0 < a.max_tokens;
       t0 += (int64_t)gridDim.x * blockDim.x * 2) {
    int32_t seq[2];
    int64_t pos[2], row[2];
    int lo = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int t = (int)t0 + k;
      seq[k] = -1;
      pos[k] = row[k] = -1;
      if (t >= n_tok) continue;
      int hi = S - 1;                             // the last sequence with tok[s] <= t
      if (k == 1 && tok[lo + 1] > t) hi = lo;     // most often the neighbour's
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tok[mid] <= t) lo = mid; else hi = mid - 1;
      }
      if (page0[lo] < 0) continue;
      const int o = held[lo];
      const int p = o + (t - tok[lo]);
      const int have = (o + kPageRows - 1) / kPageRows, col = p / kPageRows;
      int32_t* entry = a.block_table + (int64_t)lo * a.max_pages + col;
      const int page = col < have ? *entry : __ldg(a.free_pages + page0[lo] + (col - have));
      if (col >= have && p % kPageRows == 0) *entry = page;
      if (page < 0) report(a.status, CSA2_ERR_CAPACITY);
      seq[k] = lo;
      pos[k] = p;
      row[k] = page < 0 ? -1 : (int64_t)page * kPageRows + p % kPageRows;
    }
    if (t0 + 1 < a.max_tokens) {
      *reinterpret_cast<int2*>(a.q_seq + t0) = make_int2(seq[0], seq[1]);
      *reinterpret_cast<longlong2*>(a.q_pos + t0) = make_longlong2(pos[0], pos[1]);
      *reinterpret_cast<longlong2*>(a.rows + t0) = make_longlong2(row[0], row[1]);
    } else {
      a.q_seq[t0] = seq[0];
      a.q_pos[t0] = pos[0];
      a.rows[t0] = row[0];
    }
  }
}

}  // namespace
}  // namespace csa2

extern "C" size_t csa2_plan_pages_workspace(void) { return CSA2_STATUS_BYTES; }

extern "C" csa2_status_t csa2_plan_pages(int32_t num_seqs, const int32_t* old_len,
                                         const int32_t* new_len, int32_t max_tokens,
                                         int32_t* block_table, int32_t max_pages,
                                         const int32_t* free_pages, int32_t num_free,
                                         const int32_t* free_used, int32_t* free_used_out,
                                         int32_t* seq_len, int32_t* tok_start, int32_t* q_seq,
                                         int64_t* q_pos, int64_t* rows, void* workspace,
                                         size_t ws_bytes, void* stream) {
  using namespace csa2;
  if (num_seqs < 1 || max_tokens < 1 || max_tokens > (1 << 30) || max_pages < 1 || num_free < 0)
    return CSA2_ERR_INVALID_ARG;
  if (num_seqs > kPlanMaxSeqs || max_pages >= (1 << 24)) return CSA2_ERR_UNSUPPORTED;
  if (!workspace || ws_bytes < CSA2_STATUS_BYTES) return CSA2_ERR_CAPACITY;
  if (!old_len || !new_len || !block_table || (num_free > 0 && !free_pages) || !free_used ||
      !free_used_out || !seq_len || !tok_start || !q_seq || !q_pos || !rows)
    return CSA2_ERR_INVALID_ARG;
  if (seq_len == old_len || seq_len == new_len || free_used_out == free_used ||
      tok_start == old_len || tok_start == new_len)
    return CSA2_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(q_seq) | reinterpret_cast<uintptr_t>(q_pos) |
       reinterpret_cast<uintptr_t>(rows)) & 15)
    return CSA2_ERR_INVALID_ARG;
  PlanArgs a{num_seqs, old_len, new_len, max_tokens, block_table, max_pages, free_pages, num_free,
             free_used, free_used_out, seq_len, tok_start, q_seq, q_pos, rows,
             static_cast<int*>(workspace)};
  // The kernel's limit is every host thread's, so it is always set to the most that any call takes:
  // a smaller call's own size could come between another thread's setting and its launch.
  auto bytes = [](int n) { return ((size_t)n * 3 + 1) * sizeof(int32_t); };
  const size_t smem = bytes(num_seqs);
  if (smem > 40 * 1024 &&                                 // with the static part, 48 KB need no asking
      checked(cudaFuncSetAttribute(plan_pages_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   (int)bytes(kPlanMaxSeqs))) != cudaSuccess)
    return CSA2_ERR_CUDA;
  const int sms = csa2_device_sms();
  // a decode step is all latency, and a small block's barriers are short (64 sequences: 3.6 us with
  // 256 threads, 6.6 with 1,024); many sequences or tokens want the threads
  const int threads = num_seqs <= 256 && max_tokens <= 4096 ? 256 : kPlanThreads;
  const int64_t want = ((int64_t)max_tokens + 2 * threads - 1) / (2 * threads);
  const int grid = (int)(want < (sms > 0 ? sms : 1) ? want : (sms > 0 ? sms : 1));
  return launch_pdl(plan_pages_kernel, dim3(grid), dim3(threads), smem, (cudaStream_t)stream,
                    a) == cudaSuccess
             ? CSA2_OK
             : CSA2_ERR_CUDA;
}
