// Quantise + append into the paged 8-bit cache, the keys rotated on the way.
//
// The unit of work is (16-token block, head, K or V): its scale depends on all of the block's
// tokens, so one warp takes the block's new tokens (at most 16 * 128 values, in registers),
// their largest magnitude, the block's exponent, rescales the older codes if that grew, and
// writes the new ones.  A block belongs to the CTA whose window of consecutive tokens holds
// its first new token (its leader).  The window grows from 1 to 64 tokens with the batch: a
// decode token leads its own block and spreads over the GPU, a prefill fills it with two waves
// of CTAs (and up to a few CTAs more, as windows are rounded down) that each look up their tokens,
// compute their angles once for all heads, and then stream.  No two warps ever touch the same
// block.  A prefill has to move 2 bytes in and 1 out per value; what bounds it is the warps' own
// latency: 122 registers leave 16 warps per SM, which use half of the issue slots.  17,300 rotated
// tokens of 8 heads of 128 take 36.5 us (2.91 TB/s).  Decodes are a chain of look-ups: 64 take 6.3 us.
//
// A lane's item is two vectors of 8 channels of one token, chosen so that the pairs of either
// rotary layout lie inside it: neighbours, or channels i .. and i + rot / 2 .. .
#include "kv8.cuh"
#include "rope.cuh"

namespace csa2 {
namespace {

constexpr int kApThreads = 256;
constexpr int kApCtas = 2;                          // per SM
constexpr int kApWindow = 64;                       // most tokens of a CTA's window
constexpr int kApMaxD = 128;                        // most channels of a head, rotated ones too

struct AppendArgs {
  const uint16_t* x[2];                             // k, v
  int64_t stride[2];
  int num_tokens, window, heads_per_cta;
  uint8_t* codes[2];
  uint8_t* exps[2];
  int num_pages, H_kv, D;
  int num_seqs, q_per_seq, max_pages;
  const int32_t* seq_len;
  const int32_t* block_table;
  const int32_t* q_seq;
  const int32_t* tok_start;
  int* status;
  int has_rope;
  RopeArgs r;
};

struct Leader {
  int tok;                                          // its index in the window
  int page;
  int slot;                                         // its row in the page
  int count;                                        // the block's new tokens
  int64_t pos;
};

// 8 bf16
__device__ __forceinline__ void widen8(const uint4& t, float* v) {
  const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ float2 turn(float2 t, float a, float b) {
  return make_float2(a * t.x - b * t.y, b * t.x + a * t.y);
}

// Where pair p of a token stands in its row of angles.  In the vector form eight pairs belong to
// one lane: pairs 2q, 2q + 1 of all lanes lie side by side, so that the 16-byte reads of
// neighbouring lanes are conflict-free.
template <int kRope>
__device__ __forceinline__ int turn_at(int p, int half) {
  return kRope == 1 ? ((p >> 1 & 3) * (half >> 3) + (p >> 3)) * 2 + (p & 1) : p;
}

// A lane's place in every unit: two vectors of 8 channels (ea .. , eb ..) of tokens row,
// row + step, ... of the block.  kRope: 0 none, 1 the two-halves layout with rot / 2 and the offset
// multiples of 8, in which the two vectors are partners where they are rotated at all, 2 any other.
struct Place {
  int row, step;                                    // row >= 16: a lane without work
  int ea, eb;
  int turn;                                         // kRope 1: where its angles start, or -1
};
template <int kRope>
__device__ __forceinline__ Place place(const AppendArgs& a) {
  const int lane = threadIdx.x & 31, per = a.D / 16, m = lane % per, half = a.r.rot / 2;
  Place p;
  p.step = 32 / per;
  p.row = lane < p.step * per ? lane / per : kKv8Block;
  p.ea = 16 * m;
  p.eb = p.ea + 8;
  p.turn = -1;
  if constexpr (kRope == 1) {                       // rotated vectors first, then the others in order
    const int turned = half / 8;
    if (m < turned) {
      p.ea = a.r.offset + 8 * m;
      p.eb = p.ea + half;
      p.turn = 2 * m;
    } else {
      p.ea = 16 * (m - turned);
      p.eb = p.ea + 8;
      if (p.ea >= a.r.offset) p.ea += a.r.rot;
      if (p.eb >= a.r.offset) p.eb += a.r.rot;
    }
  }
  return p;
}

// the two vectors of one token, rotated; cs: its angles
template <int kRope>
__device__ __forceinline__ void rotate16(const RopeArgs& r, const uint16_t* head, const Place& pl,
                                         const float2* cs, float* v) {
  const int half = r.rot / 2;
  if constexpr (kRope == 1) {
    if (pl.turn < 0) return;
    const float2* t4 = cs + pl.turn;
#pragma unroll
    for (int q = 0; q < 4; ++q, t4 += half / 4) {
      const float4 t = *reinterpret_cast<const float4*>(t4);
#pragma unroll
      for (int i = 2 * q; i < 2 * q + 2; ++i) {
        const float2 y = turn(i & 1 ? make_float2(t.z, t.w) : make_float2(t.x, t.y), v[i], v[8 + i]);
        v[i] = y.x;
        v[8 + i] = y.y;
      }
    }
  } else if (r.interleaved) {                       // the offset is even: pairs stay inside
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      const int c = (p < 4 ? pl.ea : pl.eb - 8) + 2 * p - r.offset;
      if (c < 0 || c >= r.rot) continue;
      const float2 y = turn(cs[c / 2], v[2 * p], v[2 * p + 1]);
      v[2 * p] = y.x;
      v[2 * p + 1] = y.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int e = i < 8 ? pl.ea + i : pl.eb + i - 8, c = e - r.offset;
      if (c < 0 || c >= r.rot) continue;
      const bool first = c < half;
      const float other = __uint_as_float((uint32_t)__ldg(head + e + (first ? half : -half)) << 16);
      const float2 t = cs[first ? c : c - half];
      v[i] = first ? v[i] * t.x - other * t.y : v[i] * t.x + other * t.y;
    }
  }
}

struct Unit {
  const uint16_t* src;                              // the head of the leader's token
  int64_t stride;
  uint8_t* dst;                                     // its codes
  uint8_t* exp_at;
  int held, count;
};

// One unit by one warp; turns: the leader's row of angles.
template <int kRope>
__device__ __forceinline__ void append_unit(const AppendArgs& a, const Unit& u, const Place& pl,
                                            const float2* turns) {
  const int lane = threadIdx.x & 31, D = a.D, half = a.r.rot / 2;
  uint4 raw[4][2];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int i = pl.row + k * pl.step;
    raw[k][0] = raw[k][1] = make_uint4(0u, 0u, 0u, 0u);
    if (i < u.count) {
      const uint16_t* head = u.src + i * u.stride;
      raw[k][0] = __ldg(reinterpret_cast<const uint4*>(head + pl.ea));
      raw[k][1] = __ldg(reinterpret_cast<const uint4*>(head + pl.eb));
    }
  }
  const int was = u.held ? kv8_exp(*u.exp_at) : kKv8MinExp;
  // Rotated values are held as fp32 (a second rotation costs more than the occupancy gives);
  // others stay bf16 until they are converted.
  float rot[kRope ? 4 : 1][16];
  // the largest magnitude; a NaN is passed over
  uint32_t top = 0;                                 // magnitudes compare like their bits
  if constexpr (kRope != 0) {
    float amax = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float* v = rot[k];
      widen8(raw[k][0], v);
      widen8(raw[k][1], v + 8);
      const int i = pl.row + k * pl.step;
      if (i < u.count) rotate16<kRope>(a.r, u.src + i * u.stride, pl, turns + i * half, v);
#pragma unroll
      for (int c = 0; c < 16; ++c) amax = fmaxf(amax, fabsf(v[c]));
      asm volatile("" ::: "memory");                // one token's angles in registers at a time
    }
    top = __float_as_uint(amax);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const uint4 r = raw[k][c];
        top = __vmaxu2(top, __vmaxu2(__vmaxu2(r.x & 0x7FFF7FFFu, r.y & 0x7FFF7FFFu),
                                     __vmaxu2(r.z & 0x7FFF7FFFu, r.w & 0x7FFF7FFFu)));
      }
    top = max(top & 0xFFFFu, top >> 16) << 16;
    if (top > 0x7F800000u) {                        // a NaN among them: without the NaNs
      float amax = 0.0f;
#pragma unroll 1
      for (int k = 0; k < 4; ++k) {
        const int i = pl.row + k * pl.step;
        if (i >= u.count) break;
        for (int c = 0; c < 16; ++c) {
          const uint16_t w = u.src[i * u.stride + (c < 8 ? pl.ea + c : pl.eb + c - 8)];
          amax = fmaxf(amax, fabsf(__uint_as_float((uint32_t)w << 16)));
        }
      }
      top = __float_as_uint(amax);
    }
  }
  const float amax = __uint_as_float(__reduce_max_sync(0xffffffffu, top));
  const int now = max(was, min(kKv8MaxExp, kv8_least_exp(amax)));
  if (now > was && u.held) {                        // 16-byte vectors of the older rows
    const float f = exp2i(max(-126, was - now));
    uint4* old = reinterpret_cast<uint4*>(u.dst - (int64_t)u.held * D);
    for (int k = lane; k < u.held * (D / 16); k += 32) {
      uint4 t = old[k];
      uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float2 lo = e4m3x2_value(w[c] & 0xFFFFu), hi = e4m3x2_value(w[c] >> 16);
        w[c] = e4m3x2(lo.x * f, lo.y * f) | e4m3x2(hi.x * f, hi.y * f) << 16;
      }
      old[k] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  __syncwarp();                                     // every lane has read the old exponent
  if (lane == 0) *u.exp_at = (uint8_t)(now + kKv8Bias);
  const float f = exp2i(-now);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int i = pl.row + k * pl.step;
    if (i < u.count) {
      float v[16];
      if constexpr (kRope != 0) {
#pragma unroll
        for (int c = 0; c < 16; ++c) v[c] = rot[k][c];
      } else {
        widen8(raw[k][0], v);
        widen8(raw[k][1], v + 8);
      }
      uint32_t w[4], nan = 0;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        w[c] = e4m3x2(v[4 * c] * f, v[4 * c + 1] * f) | e4m3x2(v[4 * c + 2] * f, v[4 * c + 3] * f) << 16;
        nan |= (w[c] & 0x7F7F7F7Fu) + 0x01010101u;  // bit 7 of a byte: the NaN code
      }
      if (nan & 0x80808080u) {                      // zeros in their places
        report(a.status, CSA2_ERR_INVALID_ARG);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t is = ((w[c] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
          w[c] &= ~((is >> 7) * 0xFFu);
        }
      }
      uint8_t* dst = u.dst + i * D;
      *reinterpret_cast<uint2*>(dst + pl.ea) = make_uint2(w[0], w[1]);
      *reinterpret_cast<uint2*>(dst + pl.eb) = make_uint2(w[2], w[3]);
    }
  }
}

template <int kRope>
__global__ void __launch_bounds__(kApThreads, kApCtas) kv8_append_kernel(const __grid_constant__ AppendArgs a) {
  __shared__ Leader leaders[kApWindow];
  __shared__ int n_leaders;
  extern __shared__ __align__(16) float2 turn_smem[];             // [span][rot / 2]
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5;
  const int t0 = blockIdx.x * a.window;
  if (tid == 0) n_leaders = 0;
  __syncthreads();
  if (tid < a.window && t0 + tid < a.num_tokens) {
    Leader ld{};
    const int t = t0 + tid;
    const int s = a.q_seq ? __ldg(a.q_seq + t) : t / a.q_per_seq;
    int err = 0;
    if (s >= 0 && s < a.num_seqs) {
      const int begin = a.q_seq ? __ldg(a.tok_start + s) : s * a.q_per_seq;
      const int end = a.q_seq ? __ldg(a.tok_start + s + 1) : begin + a.q_per_seq;
      ld.pos = (int64_t)__ldg(a.seq_len + s) - end + t;
      if (begin < 0 || t < begin || t >= end || end > a.num_tokens || ld.pos < 0) {
        err = CSA2_ERR_INVALID_ARG;
      } else if (ld.pos % kKv8Block == 0 || t == begin) {
        ld.slot = (int)(ld.pos % kPageRows);
        ld.tok = tid;
        ld.count = min(kKv8Block - ld.slot % kKv8Block, end - t);
        const int64_t col = ld.pos / kPageRows;
        ld.page = col < a.max_pages ? __ldg(a.block_table + (int64_t)s * a.max_pages + col) : -1;
        bool whole = true;                          // the block's tokens all name the sequence
        if (a.q_seq)
#pragma unroll
          for (int i = 1; i < kKv8Block; ++i)
            if (i < ld.count) whole &= __ldg(a.q_seq + t + i) == s;
        if (!whole) err = CSA2_ERR_INVALID_ARG;
        else if (ld.page < 0 || ld.page >= a.num_pages) err = CSA2_ERR_CAPACITY;
        else leaders[atomicAdd(&n_leaders, 1)] = ld;        // any order: blocks are independent
      } else if (a.q_seq && __ldg(a.q_seq + t - 1) != s) {
        err = CSA2_ERR_INVALID_ARG;                 // its block's leader does not take it along
      }
    } else if (s != -1) {
      err = CSA2_ERR_INVALID_ARG;
    }
    if (err) report(a.status, err);
  }
  __syncthreads();
  const int nl = n_leaders;
  if (nl == 0) return;
  if constexpr (kRope != 0) {
    const int half = a.r.rot / 2, lane = tid & 31;
    if (a.window < kKv8Block) {                     // few tokens: all threads at each leader's
      for (int l = 0; l < nl; ++l)
        for (int k = tid; k < leaders[l].count * half; k += kApThreads) {
          const int i = k / half, p = k - i * half;
          turn_smem[(leaders[l].tok + i) * half + turn_at<kRope>(p, half)] =
              rope_turn(a.r, (double)(leaders[l].pos + i), p);
        }
    } else {
      // (cos, sin)(p + i) = (cos, sin)(p) turned by i: one sincos per leader and pair, and one for
      // each of the block's 16 steps
      float2* const first = turn_smem + (a.window + kKv8Block - 1) * half;   // [leader][pair]
      float2* const steps = first + nl * half;                               // [16][pair]
      for (int k = warp; k < nl + kKv8Block; k += kApThreads / 32) {
        const double pos = k < nl ? (double)leaders[k].pos : (double)(k - nl);
        for (int p = lane; p < half; p += 32)
          (k < nl ? first + k * half : steps + (k - nl) * half)[p] =
              k < nl ? rope_turn(a.r, pos, p) : rope_unit(a.r, pos, p);
      }
      __syncthreads();
      for (int k = warp; k < nl * kKv8Block; k += kApThreads / 32) {
        const Leader& ld = leaders[k / kKv8Block];
        const int i = k % kKv8Block;
        const float2* from = first + k / kKv8Block * half;
        if (i < ld.count)
          for (int p = lane; p < half; p += 32)
            turn_smem[(ld.tok + i) * half + turn_at<kRope>(p, half)] =
                turn(steps[i * half + p], from[p].x, from[p].y);
      }
    }
    __syncthreads();
  }
  const int D = a.D;
  const Place plain = place<0>(a), turned = place<kRope>(a);
  const int h0 = blockIdx.y * a.heads_per_cta;
  const int nh = min(a.heads_per_cta, a.H_kv - h0);
  for (int k = warp; k < nl * nh * 2; k += kApThreads / 32) {
    const int kv = k >= nl * nh, at = kv ? k - nl * nh : k, h = h0 + at % nh;   // all keys first
    const Leader ld = leaders[at / nh];
    const int64_t ph = (int64_t)ld.page * a.H_kv + h;
    Unit u;
    u.stride = kv ? a.stride[1] : a.stride[0];
    u.src = (kv ? a.x[1] : a.x[0]) + (int64_t)(t0 + ld.tok) * u.stride + (int64_t)h * D;
    u.dst = (kv ? a.codes[1] : a.codes[0]) + (ph * kPageRows + ld.slot) * D;
    u.exp_at = (kv ? a.exps[1] : a.exps[0]) + ph * kKv8Blocks + ld.slot / kKv8Block;
    u.held = ld.slot % kKv8Block;                           // the block's older tokens
    u.count = ld.count;
    if (kRope == 0 || kv) append_unit<0>(a, u, plain, nullptr);
    else append_unit<kRope>(a, u, turned, turn_smem + ld.tok * (a.r.rot / 2));
  }
}

}  // namespace
}  // namespace csa2

extern "C" size_t csa2_kv8_append_workspace(void) { return CSA2_STATUS_BYTES; }

extern "C" csa2_status_t csa2_kv8_append(const uint16_t* k, int64_t k_stride, const uint16_t* v,
                                         int64_t v_stride, int32_t num_tokens, csa2_kv8_t cache,
                                         csa2_seqs_t seqs, const int32_t* tok_start,
                                         const csa2_rope_t* rope, void* workspace, size_t ws_bytes,
                                         void* stream) {
  using namespace csa2;
  if (num_tokens < 0 || seqs.num_seqs < 1) return CSA2_ERR_INVALID_ARG;
  const csa2_status_t bad = kv8_check(cache);
  if (bad != CSA2_OK) return bad;
  if (num_tokens > (1 << 30)) return CSA2_ERR_UNSUPPORTED;
  const int64_t row = (int64_t)cache.H_kv * cache.D;
  if (k_stride < row || v_stride < row || k_stride % 8 || v_stride % 8) return CSA2_ERR_INVALID_ARG;
  if (!workspace || ws_bytes < CSA2_STATUS_BYTES) return CSA2_ERR_CAPACITY;
  if ((seqs.q_seq == nullptr) != (tok_start == nullptr)) return CSA2_ERR_INVALID_ARG;
  if (!seqs.q_seq &&
      (seqs.q_per_seq < 1 || (int64_t)seqs.num_seqs * seqs.q_per_seq != num_tokens))
    return CSA2_ERR_INVALID_ARG;
  AppendArgs a{};
  if (rope) {
    const csa2_status_t st = rope_args(rope, &a.r);
    if (st != CSA2_OK) return st;
    if ((int64_t)a.r.offset + a.r.rot > cache.D) return CSA2_ERR_INVALID_ARG;
    a.has_rope = 1;
  }
  if (num_tokens == 0) return CSA2_OK;
  if (!k || !v || !seqs.seq_len || !seqs.block_table || seqs.max_pages < 1 ||
      ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 15) ||
      !kv8_pointers_ok(cache))
    return CSA2_ERR_INVALID_ARG;
  a.x[0] = k;
  a.x[1] = v;
  a.stride[0] = k_stride;
  a.stride[1] = v_stride;
  a.num_tokens = num_tokens;
  a.codes[0] = cache.k;
  a.codes[1] = cache.v;
  a.exps[0] = cache.k_exp;
  a.exps[1] = cache.v_exp;
  a.num_pages = cache.num_pages;
  a.H_kv = cache.H_kv;
  a.D = cache.D;
  a.num_seqs = seqs.num_seqs;
  a.q_per_seq = seqs.q_per_seq;
  a.max_pages = seqs.max_pages;
  a.seq_len = seqs.seq_len;
  a.block_table = seqs.block_table;
  a.q_seq = seqs.q_seq;
  a.tok_start = tok_start;
  a.status = static_cast<int*>(workspace);
  // Two waves of CTAs before windows and head groups grow: with one wave the CTA with the most
  // blocks decides (17,300 tokens of 8 heads: 43 us; two waves 36, four waves of 16-token windows,
  // whose look-ups and angles serve fewer tokens, 65).  Windows and head groups are rounded down, so
  // the grid is at least that: 597 CTAs for those tokens on 592 places.
  const int64_t want = 2 * kApCtas * (int64_t)(csa2_device_sms() > 0 ? csa2_device_sms() : 148);
  const int64_t units = (int64_t)num_tokens * cache.H_kv;
  a.window = (int)(units / want < 1 ? 1 : units / want > kApWindow ? kApWindow : units / want);
  if (a.window > kKv8Block && (int64_t)num_tokens / a.window < want)
    a.window = (int)(num_tokens / want < kKv8Block ? kKv8Block : num_tokens / want);
  const int64_t gx = ((int64_t)num_tokens + a.window - 1) / a.window;
  int64_t hpc = gx * cache.H_kv / want;
  a.heads_per_cta = (int)(hpc < 1 ? 1 : hpc > cache.H_kv ? cache.H_kv : hpc);
  const int gy = (cache.H_kv + a.heads_per_cta - 1) / a.heads_per_cta;
  const int mode = !a.has_rope ? 0
                   : !a.r.interleaved && (a.r.rot / 2) % 8 == 0 && a.r.offset % 8 == 0 ? 1 : 2;
  auto* kernel = mode == 0   ? kv8_append_kernel<0>
                 : mode == 1 ? kv8_append_kernel<1>
                             : kv8_append_kernel<2>;
  // Angles of the window's reach, of its leaders and of a block's steps.  The kernel's limit is
  // every host thread's, so it is always set to the most that any call takes.
  auto bytes = [](int window, int rot) {
    return (size_t)(window + kKv8Block - 1 + window + kKv8Block) * (rot / 2) * sizeof(float2);
  };
  const size_t smem = mode ? bytes(a.window, a.r.rot) : 0;
  if (smem > 40 * 1024 &&                                 // with the static part, 48 KB need no asking
      checked(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   (int)bytes(kApWindow, kApMaxD))) != cudaSuccess)
    return CSA2_ERR_CUDA;
  return launch_pdl(kernel, dim3((unsigned)gx, gy), dim3(kApThreads), smem,
                    (cudaStream_t)stream, a) == cudaSuccess
             ? CSA2_OK
             : CSA2_ERR_CUDA;
}
