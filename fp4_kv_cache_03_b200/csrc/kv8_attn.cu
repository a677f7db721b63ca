// Causal attention over the paged 8-bit cache, for few query rows per KV head (decoding).
//
// Bound by HBM: every visible key and value byte is read once per KV head and serves all
// G = H / H_kv heads and all queries of its job.  The codes are never converted: a page's
// 128 x D tile goes by TMA into shared memory and straight into tcgen05.mma kind::f8f6f4 as
// the A operand, for
//   S^T[key, row] = K[key, :] . Q[row, :]        (M = 128 keys,     K-major)
//   O^T[d, row]  += V^T[d, key] . P^T[key, row]  (M = 128 channels, the same layout MN-major)
// What has to stay precise is split into E4M3 terms instead, on the narrow side:
//   Q (bf16, 8 significant bits), scaled per row by a power of two so that its largest is in
//     (224, 448], is hi + lo of 4 bits each: two MMAs into one accumulator;
//   P = p0 + p1 / 2^4 + p2 / 2^8 + p3 / 2^15, each remainder scaled by 16, 16 and 128 and rounded
//     again (none passes 256): a weight is off by at most 2^-11 of itself plus 2^-26 of the row's
//     largest, and one of 2^-29 of it is not lost yet.  With three terms those under 2^-22 all were,
//     and tens of thousands of them beside one large weight make up a visible part of the sum.  The
//     four accumulate in columns of their own (one MMA of 4R columns) and are added at the end.
// An MMA here costs the read of its A operand (a 128 x 32-byte slice), whatever its N, so the
// terms are nearly free.  Key scales multiply S; value scales 2^e add e to the exponent's
// argument, x_j + e_j, and the running reference is the maximum of that sum, so the largest
// weight is always near the top of E4M3's range; the softmax's own sum takes w_j * 2^-e_j.
//
// One key per TMEM lane makes the maximum over keys a reduction over threads.  It is only taken
// when some weight would leave [0, 16] times the reference (every first tile, then rarely): one
// barrier with an OR finds that out.
//
// Warp roles: softmax (4 warps), TMA producer, MMA issuer, 2 warps that fetch and
// split the next job's Q.  K and V tiles alternate in a ring of 16 KB units in the order that
// the MMAs consume them: K0 K1 V0 K2 V1 ..., so S of tile t+1 runs under the softmax of tile t.
//
// One token over 1,048,576 tokens, 64 heads on 8 of 128: 341 to 346 us (6.2 to 6.3 TB/s); 64 ragged
// decodes over 485,000 tokens: 208 us.
#include <cudaTypedefs.h>

#include "kv8_attn.cuh"

namespace csa2 {
namespace {

constexpr int kTerms = 4;                      // of P
// what is left of a weight behind term k is scaled by this before it is rounded to term k + 1
__device__ __forceinline__ constexpr float kv8_step(int k) { return k < 2 ? 16.0f : 128.0f; }
constexpr float kTopLog2 = 4.0f;               // a fresh reference's weight is 2^4 ...
constexpr float kGrowLog2 = 4.0f;              // ... and may grow to 2^8 before a rescale

constexpr int kv8_ctas_per_sm(int rows) { return rows == kPrefillRows ? 1 : rows == 8 ? 3 : 2; }
constexpr uint32_t kv8_cols(uint32_t n) {
  return n <= 64 ? 64 : n <= 128 ? 128 : n <= 256 ? 256 : 512;
}

// R: rows (queries x heads of one KV head) per job; kUnits: ring units
template <int R, int kUnits>
struct DecGeo {
  static constexpr int kSmWarps = 4;
  static constexpr int kThreads = kSmWarps * 32 + 128;
  // per SM: each tile is a chain of waits (about 3,600 cycles), so CTAs beside one another keep
  // the loads going; a ring of 3 units each is enough then.  64 ragged decodes, 1.0 GB: 203 us
  // with 3 CTAs of 3 units, 214 with 2 of 5.  16 rows need more registers than 3 leave.
  static constexpr int kCtas = kv8_ctas_per_sm(R);
  static constexpr int N = R < 16 ? 16 : R;                 // columns of S^T
  static constexpr int NP = (kTerms * R + 15) / 16 * 16;    // columns of O^T
  static constexpr uint32_t kTmemO = 2 * N;
  static constexpr uint32_t kTmemCols = kv8_cols(2 * N + NP);
  static constexpr uint32_t kP = NP * 128;
  static constexpr uint32_t kQ = N * 128;
  static constexpr uint32_t kOffP = kUnits * kUnit;
  static constexpr uint32_t kOffQ = kOffP + 2 * kP;
  static constexpr uint32_t kSmem = 1024 + kOffQ + 4 * kQ;
};

struct TileInfo {
  uint2 kx, vx;                                // 8 + 8 scale bytes
  int ok;                                      // the tile was loaded
};

template <int R, int kUnits>
struct DecSmem {
  using G = DecGeo<R, kUnits>;
  uint64_t full[kUnits], empty[kUnits], info_full[kInfo];
  uint64_t s_full[2], s_empty[2], p_full[2], p_empty[2], q_full[2], q_empty[2], drain;
  int64_t red64[G::kThreads / 32];
  Kv8Share share;
  uint32_t tmem_base;
  int abort;
  TileInfo info[kInfo];
  alignas(16) float row_factor[2][R];          // softmax_scale * log2(e) * 2^e of the Q row
  alignas(16) int row_pos[2][R];               // the row's query position; -1: no row
  alignas(16) float m_ref[R];
  alignas(16) float alpha[R];
  alignas(16) float red[4][R];
};

__device__ __forceinline__ bool group_any(int id, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %1, 0;\n\t"
      "barrier.cta.red.or.pred p, %2, 128, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)p), "r"(id)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void group_sync(int id) {
  asm volatile("barrier.cta.sync %0, 128;" ::"r"(id) : "memory");
}
// fp32 order as signed integers (a NaN is above everything)
__device__ __forceinline__ int order_int(float x) {
  const int i = __float_as_int(x);
  return i ^ ((i >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float from_order(int i) {
  return __int_as_float(i ^ ((i >> 31) & 0x7FFFFFFF));
}
template <int R, int kUnits>
__global__ void __launch_bounds__(DecGeo<R, kUnits>::kThreads, DecGeo<R, kUnits>::kCtas)
    kv8_decode_kernel(const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const Kv8AttnArgs a) {
  using G = DecGeo<R, kUnits>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ DecSmem<R, kUnits> sm;
  uint8_t* base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort = &sm.abort;
  const int kProducer = G::kSmWarps, kIssuer = kProducer + 1, kSplit = kProducer + 2;

  if (tid == 0) {
    for (int i = 0; i < kUnits; ++i) { mbar_init(&sm.full[i], 1); mbar_init(&sm.empty[i], 1); }
    for (int i = 0; i < kInfo; ++i) mbar_init(&sm.info_full[i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.s_empty[i], G::kSmWarps);
      mbar_init(&sm.p_full[i], G::kSmWarps);
      mbar_init(&sm.p_empty[i], 1);
      mbar_init(&sm.q_full[i], 2);
      mbar_init(&sm.q_empty[i], 1 + G::kSmWarps);
    }
    mbar_init(&sm.drain, 1);
    sm.abort = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == kIssuer) { tmem_alloc(&sm.tmem_base, G::kTmemCols); tmem_relinquish(); }
  // rows of Q that pad R to the MMA's 16 stay zero
  if constexpr (G::N > R)
    for (int i = tid; i < 4 * (G::N - R) * 8; i += G::kThreads)
      *reinterpret_cast<uint4*>(base + G::kOffQ + i / ((G::N - R) * 8) * G::kQ + R * 128 +
                                i % ((G::N - R) * 8) * 16) = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  pdl_wait();
  kv8_share(a.b, blockIdx.x, gridDim.x, sm.red64, &sm.share, blockIdx.x == 0 ? a.status : nullptr);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // only now: a dependent kernel must not take tensor memory that this CTA still waits for
  pdl_trigger();
  const uint32_t tmem = sm.tmem_base;
  const int T = (int)(sm.share.end - sm.share.begin);    // key tiles of this CTA
  const int Hkv = a.b.H_kv;

  if (warp == kProducer) {
    // ------------------------------ pages -> ring ------------------------------
    Kv8Walk w;
    w.start(a.b, sm.share);
    int kb = 0;                                // the batch of 32 tiles whose pages the lanes hold
    bool fresh = true;
    int z = -1;
    uint2 kx = make_uint2(0, 0), vx = kx;
    int at = w.kt;                             // next tile of the job
    auto fetch = [&]() -> int {                // next tile's page row, or -1
      if (!fresh && at == w.kt_end) {
        w.next(a.b);
        at = w.kt;
        fresh = true;
      }
      if (fresh || at - kb == 32) {
        kb = at;
        fresh = false;
        z = -1;
        const int t = at + lane;
        if (t < w.kt_end && w.tile.p0 + w.tile.nq > 0) {
          const int page = __ldg(a.b.block_table + (int64_t)w.s * a.b.max_pages + w.tile.kt0 + t);
          if (page < 0 || page >= a.num_pages) {
            report(a.status, CSA2_ERR_CAPACITY);
          } else {
            z = page * Hkv + w.h;
            kx = __ldg(reinterpret_cast<const uint2*>(a.k_exp) + z);
            vx = __ldg(reinterpret_cast<const uint2*>(a.v_exp) + z);
          }
        }
      }
      return __shfl_sync(0xffffffffu, z, at - kb);
    };
    auto tell = [&](int g) {                   // its scales, once its keys are on their way
      if (lane == at - kb) sm.info[g % kInfo] = TileInfo{kx, vx, z >= 0};
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.info_full[g % kInfo]);
      ++at;
    };
    int unit = 0, round = 0;
    uint32_t filled = 0, filled_parity = 0;    // units filled, and the phase of the latest fill
    bool ok = true;
    auto issue = [&](const CUtensorMap* tm, int row) {
      if (lane == 0) {
        ok = ok && kv8_wait(&sm.empty[unit], (round & 1) ^ 1, abort, a.status, a.wait_ns);
        if (ok) {
          if (row >= 0) {
            mbar_arrive_expect_tx(&sm.full[unit], kUnit);
            tma_load_3d(base + unit * kUnit, tm, 0, 0, row, &sm.full[unit]);
          } else {
            mbar_arrive(&sm.full[unit]);
          }
          filled |= 1u << unit;
          filled_parity = (filled_parity & ~(1u << unit)) | (uint32_t)(round & 1) << unit;
        }
      }
      if (++unit == kUnits) { unit = 0; ++round; }
    };
    if (T > 0) {
      int cur = fetch();
      issue(&tm_k, cur);
      tell(0);
      for (int t = 0; t < T; ++t) {
        int nxt = -1;
        if (t + 1 < T) {
          nxt = fetch();
          issue(&tm_k, nxt);
          tell(t + 1);
        }
        issue(&tm_v, cur);
        cur = nxt;
        ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
        if (!ok) break;
      }
      // no load of this CTA may still be landing when it exits
      if (lane == 0)
        for (int i = 0; i < kUnits; ++i)
          if (filled & (1u << i)) mbar_drain(&sm.full[i], (filled_parity >> i) & 1u);
    }
  } else if (warp == kIssuer) {
    // ------------------------------ MMAs ------------------------------
    if (T > 0) {
      const uint32_t leader = elect_one();
      const uint32_t id_s = idesc_e4m3(128, G::N);
      const uint32_t id_o = idesc_e4m3(128, G::NP) | (1u << 15);    // A = V^T is MN-major
      const int ksteps = (a.D + 31) / 32;
      // descriptors; the address field counts 16 bytes
      const uint64_t su0 = sdesc_sw128(smem_u32(base), 16, 1024);
      const uint64_t sp0 = sdesc_sw128(smem_u32(base + G::kOffP), 16, 1024);
      const uint64_t sq0 = sdesc_sw128(smem_u32(base + G::kOffQ), 16, 1024);
      Kv8Walk w;
      w.start(a.b, sm.share);
      int unit = 0, round = 0, job = 0, at = w.kt;
      bool ok = true;
      auto wait_unit = [&]() {
        ok = ok && kv8_wait_warp(&sm.full[unit], round & 1, abort, a.status, a.wait_ns);
      };
      auto next_unit = [&]() { if (++unit == kUnits) { unit = 0; ++round; } };
      bool first_prev = true;                  // tile t - 1 began its job
      for (int t = 0; t <= T && ok; ++t) {
        bool first = false;
        if (t < T) {
          if (at == w.kt_end) {
            w.next(a.b);
            at = w.kt;
            ++job;
          }
          first = at == w.kt;
          wait_unit();
          if (first)
            ok = ok && kv8_wait_warp(&sm.q_full[job & 1], (job >> 1) & 1, abort, a.status, a.wait_ns);
          ok = ok && kv8_wait_warp(&sm.s_empty[t & 1], ((t >> 1) & 1) ^ 1, abort, a.status, a.wait_ns);
          if (!ok) break;
          tc_fence_after();
          const uint64_t ad = su0 + (uint32_t)unit * (kUnit >> 4);
          const uint64_t bd = sq0 + (uint32_t)(job & 1) * (2 * G::kQ >> 4);
          const uint32_t d = tmem + (t & 1) * G::N;
#pragma unroll
          for (int k = 0; k < 4; ++k)          // 32 channels, 32 bytes each
            if (k < ksteps) {
              warp_umma_e4m3(leader, d, ad + k * 2, bd + k * 2, id_s, k > 0);
              warp_umma_e4m3(leader, d, ad + k * 2, bd + (G::kQ >> 4) + k * 2, id_s, 1);
            }
          warp_commit(leader, &sm.empty[unit]);
          warp_commit(leader, &sm.s_full[t & 1]);
          ++at;
          if (at == w.kt_end) warp_commit(leader, &sm.q_empty[job & 1]);
          next_unit();
        }
        if (t > 0) {
          const int p = (t - 1) & 1;
          wait_unit();
          ok = ok && kv8_wait_warp(&sm.p_full[p], ((t - 1) >> 1) & 1, abort, a.status, a.wait_ns);
          if (!ok) break;
          tc_fence_after();
          const uint64_t ad = su0 + (uint32_t)unit * (kUnit >> 4);
          const uint64_t bd = sp0 + (uint32_t)p * (G::kP >> 4);
#pragma unroll
          for (int k = 0; k < 4; ++k)          // 32 keys each
            warp_umma_e4m3(leader, tmem + G::kTmemO, ad + k * (4096 >> 4), bd + k * 2, id_o,
                           k > 0 || !first_prev);
          warp_commit(leader, &sm.empty[unit]);
          warp_commit(leader, &sm.p_empty[p]);
          next_unit();
        }
        first_prev = first;
      }
      // every MMA this warp issued has completed before the CTA frees TMEM and exits
      warp_commit(leader, &sm.drain);
      mbar_drain(&sm.drain, 0);
      __syncwarp();
    }
  } else if (warp >= kSplit) {
    // ------------------------------ Q -> two E4M3 terms ------------------------------
    const int wq = warp - kSplit;
    Kv8Desc d{0, 0, 0, 0, 0};
    if (T > 0) {
      Kv8Walk w;
      w.start(a.b, sm.share);
      for (int job = 0; !w.done(); ++job, w.next(a.b)) {
        const int jb = job & 1;
        if (!w.begins()) d.head_ends = w.ends();
        if (w.begins() && !w.ends())
          d = Kv8Desc{1, d.head_ends, w.seq.q0 + w.i * a.b.QT, w.tile.nq * a.b.G, w.h};
        if (lane == 0) kv8_wait(&sm.q_empty[jb], ((job >> 1) & 1) ^ 1, abort, a.status, a.wait_ns);
        __syncwarp();
        uint8_t* qb = base + G::kOffQ + jb * 2 * G::kQ;
        const int rows = w.tile.nq * a.b.G;
        const uint16_t* q0 = a.q + (int64_t)(w.seq.q0 + w.i * a.b.QT) * a.q_stride +
                             (int64_t)w.h * a.b.G * a.D + lane * 4;
        constexpr int kBatch = 4;
#pragma unroll 1
        for (int r0 = wq; r0 < R; r0 += 2 * kBatch) {
          uint2 x[kBatch];
#pragma unroll
          for (int j = 0; j < kBatch; ++j) {
            const int r = r0 + 2 * j;
            x[j] = make_uint2(0u, 0u);
            if (r < rows && lane * 4 < a.D)
              x[j] = __ldg(reinterpret_cast<const uint2*>(q0 + (r / a.b.G) * a.q_stride +
                                                          (r % a.b.G) * (int64_t)a.D));
          }
#pragma unroll
          for (int j = 0; j < kBatch; ++j) {
            const int r = r0 + 2 * j;
            float v[4] = {__uint_as_float(x[j].x << 16), __uint_as_float(x[j].x & 0xFFFF0000u),
                          __uint_as_float(x[j].y << 16), __uint_as_float(x[j].y & 0xFFFF0000u)};
            const uint32_t top = __reduce_max_sync(
                0xffffffffu, max(max(x[j].x & 0x7FFFu, x[j].x >> 16 & 0x7FFFu),
                                 max(x[j].y & 0x7FFFu, x[j].y >> 16 & 0x7FFFu)));
            const float amax = __uint_as_float(top << 16);
            const int e = max(-120, min(119, kv8_least_exp(amax)));
            const float f = exp2i(-e);
            uint32_t hi = 0, lo = 0;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const float p = v[2 * c] * f, s = v[2 * c + 1] * f;
              const uint32_t h2 = e4m3x2(p, s);
              const float2 hv = e4m3x2_value(h2);
              hi |= h2 << (16 * c);
              lo |= e4m3x2(p - hv.x, s - hv.y) << (16 * c);
            }
            *reinterpret_cast<uint32_t*>(qb + sw128(r, lane * 4)) = hi;
            *reinterpret_cast<uint32_t*>(qb + G::kQ + sw128(r, lane * 4)) = lo;
            if (lane == 0) {
              // a row with an infinity or a NaN gives NaN, not a saturated answer
              const float sc = top >= 0x7F80u ? __int_as_float(0x7FC00000) : a.scale_log2 * exp2i(e);
              sm.row_factor[jb][r] = r < rows ? sc : 0.0f;
              sm.row_pos[jb][r] = r < rows ? w.tile.p0 + r / a.b.G : -1;
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.q_full[jb]);
      }
    }
    if (wq == 0 && lane == 0) a.desc[blockIdx.x] = d;
  } else {
    // ------------------------------ softmax ------------------------------
    constexpr int CW = R;
    const int quad = warp, key = quad * 32 + lane;       // also the channel of O^T
    const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
    constexpr int bar = 1;
    auto wait = [&](uint64_t* b, uint32_t parity) {
      if (lane == 0) kv8_wait(b, parity, abort, a.status, a.wait_ns);
      __syncwarp();
    };
    int g = 0;
    Kv8Walk w;
    if (T > 0) w.start(a.b, sm.share);
    else w.left = 0;
    for (int job = 0; !w.done(); ++job, w.next(a.b)) {
      const int jb = job & 1;
      wait(&sm.q_full[jb], (job >> 1) & 1);
      float sum[CW];
#pragma unroll
      for (int c = 0; c < CW; ++c) sum[c] = 0.0f;
      const int p_first = w.tile.p0, p_last = w.tile.p0 + w.tile.nq - 1;
      for (int kt = w.kt; kt < w.kt_end; ++kt, ++g) {
        const int b = g & 1;
        const uint32_t k2 = (uint32_t)(g >> 1) & 1u;
        wait(&sm.info_full[g % kInfo], (uint32_t)(g / kInfo) & 1u);
        const bool loaded = sm.info[g % kInfo].ok != 0;
        const int blk = key / kKv8Block;
        const int ke = kv8_exp(reinterpret_cast<const uint8_t*>(&sm.info[g % kInfo].kx)[blk]);
        const int ve = kv8_exp(reinterpret_cast<const uint8_t*>(&sm.info[g % kInfo].vx)[blk]);
        const float kf = exp2i(ke), vef = (float)ve, vinv = exp2i(-ve);
        const int j0 = (w.tile.kt0 + kt) * kPageRows, j = j0 + key;
        const bool whole = loaded && j0 + kPageRows - 1 <= p_first &&
                           (!a.b.window || j0 > p_last - a.b.window);
        wait(&sm.s_full[b], k2);
        tc_fence_after();
        float x[CW];
#pragma unroll
        for (int c = 0; c < CW; c += 8) tmem_ldn<8>(tmem + lane_base + b * G::N + c, x + c);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.s_empty[b]);
        bool over = kt == w.kt;
#pragma unroll
        for (int c = 0; c < CW; ++c) {
          x[c] = fmaf(x[c], sm.row_factor[jb][c] * kf, vef);
          if (!whole) {
            const int t = sm.row_pos[jb][c];
            if (!loaded || j > t || (a.b.window && j <= t - a.b.window)) x[c] = -INFINITY;
          }
          over |= x[c] > sm.m_ref[c] + kGrowLog2;
        }
        if (group_any(bar, over)) {
          // exact maxima: per warp, then over the four warps of the group
          float mine = -INFINITY;
#pragma unroll
          for (int c = 0; c < CW; ++c) {
            const int m = __reduce_max_sync(0xffffffffu, order_int(x[c]));
            if (lane == c) mine = from_order(m);
          }
          if (lane < CW) sm.red[quad][lane] = mine;
          group_sync(bar);
          const int c = quad * 32 + lane;
          if (c < CW) {
            const float old = kt == w.kt ? -INFINITY : sm.m_ref[c];
            float m = old;
#pragma unroll
            for (int k = 0; k < 4; ++k) m = fmaxf(m, sm.red[k][c]);
            sm.alpha[c] = old == -INFINITY ? 0.0f : ex2(old - m);
            sm.m_ref[c] = m;
          }
          group_sync(bar);
#pragma unroll
          for (int k = 0; k < CW; ++k) sum[k] *= sm.alpha[k];
          if (kt > w.kt) {
            wait(&sm.p_empty[(g - 1) & 1], (uint32_t)((g - 1) >> 1) & 1u);
            tc_fence_after();
#pragma unroll 1
            for (int part = 0; part < kTerms; ++part)
#pragma unroll 1
              for (int k = 0; k < CW; k += 8) {
                float o[8];
                const uint32_t at = tmem + lane_base + G::kTmemO + part * R + k;
                tmem_ldn<8>(at, o);
#pragma unroll
                for (int q = 0; q < 8; ++q) o[q] *= sm.alpha[k + q];
                tmem_stn<8>(at, o);
              }
            tmem_wait_st();
          }
        }
        if (!whole) {
          // what lies behind the last key or in a page that is not there must not meet a zero
          // weight as a NaN: clear the value row
          const bool clear = !loaded || j > p_last;
          if (__any_sync(0xffffffffu, clear)) {
            const int n = g + 1 < T ? 2 * g + 2 : 2 * T - 1;   // the value tile's place in the ring
            wait(&sm.full[n % kUnits], (uint32_t)(n / kUnits) & 1u);
            if (clear && !*abort) {
              uint4* row = reinterpret_cast<uint4*>(base + (n % kUnits) * kUnit + key * 128);
#pragma unroll
              for (int k = 0; k < 8; ++k) row[k] = make_uint4(0u, 0u, 0u, 0u);
            }
          }
        }
        wait(&sm.p_empty[b], k2 ^ 1u);
        uint8_t* pb = base + G::kOffP + b * G::kP;
#pragma unroll
        for (int c = 0; c < CW; c += 2) {
          float p[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float m = sm.m_ref[c + k];
            p[k] = ex2(x[c + k] - ((m == -INFINITY ? 0.0f : m) - kTopLog2));
            sum[c + k] = fmaf(p[k], vinv, sum[c + k]);
          }
          // behind the first term 11 bits of the rest are enough for the other three, and two
          // columns go in one register
          uint32_t term = e4m3x2(p[0], p[1]);
          const float2 v0 = e4m3x2_value(term);
          __half2 rest = __floats2half2_rn((p[0] - v0.x) * kv8_step(0), (p[1] - v0.y) * kv8_step(0));
#pragma unroll
          for (int k = 0; k < kTerms; ++k) {
            pb[sw128(k * R + c, key)] = (uint8_t)term;
            pb[sw128(k * R + c + 1, key)] = (uint8_t)(term >> 8);
            if (k == kTerms - 1) break;
            if (k > 0) rest = __hmul2(__hsub2(rest, e4m3x2_half2(term)), __float2half2_rn(kv8_step(k)));
            term = e4m3x2(rest);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full[b]);
      }
      // ---- the job's rows: sums over keys, then O / sum or a partial ----
#pragma unroll
      for (int c = 0; c < CW; ++c) {
        float s = sum[c];
#pragma unroll
        for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        if (lane == 0) sm.red[quad][c] = s;
      }
      group_sync(bar);
      wait(&sm.p_empty[(g - 1) & 1], (uint32_t)((g - 1) >> 1) & 1u);
      tc_fence_after();
      const bool final = w.begins() && w.ends();
      const int slot = 2 * blockIdx.x + (w.begins() ? 1 : 0);
      const int rows = w.tile.nq * a.b.G;
      const int q_row = w.seq.q0 + w.i * a.b.QT;
#pragma unroll 1
      for (int k = 0; k < CW; k += 8) {
        float o[kTerms][8];
#pragma unroll
        for (int part = 0; part < kTerms; ++part)
          tmem_ldn<8>(tmem + lane_base + G::kTmemO + part * R + k, o[part]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = k + i;
          if (r >= rows) continue;
          float v = o[kTerms - 1][i];
#pragma unroll
          for (int k = kTerms - 2; k >= 0; --k) v = fmaf(v, 1.0f / kv8_step(k), o[k][i]);
          const float l = (sm.red[0][r] + sm.red[1][r]) + (sm.red[2][r] + sm.red[3][r]);
          if (final) {
            const int64_t hrow = (int64_t)(q_row + r / a.b.G) * a.H + w.h * a.b.G + r % a.b.G;
            if (key < a.D)
              reinterpret_cast<__nv_bfloat16*>(a.out)[hrow * a.D + key] =
                  __float2bfloat16_rn(l == 0.0f ? 0.0f : v / l);
            if (key == 0 && a.lse)
              a.lse[hrow] = l == 0.0f ? -INFINITY
                                      : (sm.m_ref[r] - kTopLog2 + lg2(l)) * 0.6931471805599453f;
          } else {
            if (key < a.D) a.part_o[((int64_t)slot * R + r) * 128 + key] = v;
            if (key == 0) a.part_ml[slot * R + r] = make_float2(sm.m_ref[r] - kTopLog2, l);
          }
        }
      }
      tc_fence_before();
      group_sync(bar);                                   // red and m_ref have been read
      if (lane == 0) mbar_arrive(&sm.q_empty[jb]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kIssuer) {
    tc_fence_after();
    tmem_dealloc(tmem, G::kTmemCols);
  }
}

// Joins the partials of the jobs that several CTAs share: blocks (c, .) those of the job that
// CTA c began.  kPer warps per row, 4 channels per lane: the splits' weights 2^(m - max), one
// lane per split, then their sum, every kPer-th split by each warp (8 for a decode's few rows of
// many splits, 1 for a prefill's many rows of two or three).
constexpr int kMergeWarps = 8, kMergeBlocks = 8;           // warps of a block; most blocks per c
template <int kPer>
__global__ void __launch_bounds__(kMergeWarps * 32)
    kv8_merge_kernel(int R, int ctas, int H, int G, int D, const Kv8Desc* desc, const float* part_o,
                     const float2* part_ml, uint16_t* out, float* lse) {
  constexpr int kRows = kMergeWarps / kPer;
  __shared__ float4 part[kPer > 1 ? kMergeWarps : 1][32];
  pdl_trigger();
  pdl_wait();
  const int c = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp % kPer;
  const bool ends = c + 1 + lane < ctas && desc[c + 1 + lane].head_ends;
  const Kv8Desc d = desc[c];
  if (!d.tail || (int)blockIdx.y * kRows >= d.rows) return;
  int last = ctas - 1;                                     // the CTA in which the job ends
  uint32_t who = __ballot_sync(0xffffffffu, ends);
  for (int k = c + 1; k < ctas; k += 32) {
    if (k > c + 1) who = __ballot_sync(0xffffffffu, k + lane < ctas && desc[k + lane].head_ends);
    if (who) {
      last = k + __ffs(who) - 1;
      break;
    }
  }
  const int n = last - c + 1;                              // splits: the tail of c, heads after it
  for (int r0 = blockIdx.y * kRows; r0 < d.rows; r0 += gridDim.y * kRows) {
    const int r = r0 + warp / kPer;                        // a row past the job's: nothing written
    const bool there = r < d.rows;
    auto slot = [&](int k) { return (int64_t)(2 * (c + k) + (k == 0)) * R + r; };
    auto piece = [&](int k) {
      return lane * 4 < D && there
                 ? *reinterpret_cast<const float4*>(part_o + slot(k) * 128 + lane * 4)
                 : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    };
    constexpr int kAhead = kPer > 1 ? 32 / kPer : 2;       // pieces fetched beside the weights
    float4 ahead[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int k = sub + j * kPer;
      if (k < n) ahead[j] = piece(k);
    }
    float m = -INFINITY;
    for (int k = lane; k < n && there; k += 32) m = fmaxf(m, part_ml[slot(k)].x);
#pragma unroll
    for (int s = 16; s; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
    float l = 0.0f;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int k0 = 0; k0 < n; k0 += 32) {
      float f = 0.0f;
      if (k0 + lane < n && there) {
        const float2 ml = part_ml[slot(k0 + lane)];
        f = ml.x == -INFINITY ? 0.0f : ex2(ml.x - m);
        l += f * ml.y;
      }
      auto take = [&](int k, const float4& o) {
        const float wk = __shfl_sync(0xffffffffu, f, k);
        acc.x = fmaf(o.x, wk, acc.x);
        acc.y = fmaf(o.y, wk, acc.y);
        acc.z = fmaf(o.z, wk, acc.z);
        acc.w = fmaf(o.w, wk, acc.w);
      };
      int k = sub;
      if (k0 == 0) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j, k += kPer)
          if (k < n) take(k, ahead[j]);
      }
#pragma unroll 4
      for (; k < min(32, n - k0); k += kPer) take(k, piece(k0 + k));
    }
#pragma unroll
    for (int s = 16; s; s >>= 1) l += __shfl_xor_sync(0xffffffffu, l, s);
    if constexpr (kPer > 1) {
      part[warp][lane] = acc;
      __syncthreads();
      if (sub == 0)
#pragma unroll
        for (int k = 1; k < kPer; ++k) {
          const float4 o = part[warp + k][lane];
          acc.x += o.x;
          acc.y += o.y;
          acc.z += o.z;
          acc.w += o.w;
        }
      __syncthreads();
    }
    if (sub > 0 || !there) continue;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const int64_t hrow = (int64_t)(d.q_row0 + r / G) * H + d.h * G + r % G;
    if (lane * 4 < D) {
      const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
      const __nv_bfloat162 hi = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
      *reinterpret_cast<uint2*>(out + hrow * D + lane * 4) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    }
    if (lane == 0 && lse) lse[hrow] = l == 0.0f ? -INFINITY : (m + lg2(l)) * 0.6931471805599453f;
  }
}

constexpr int kMaxCtas = 1024;
PFN_cuTensorMapEncodeTiled_v12000 kv8_encode_fn() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult qr;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &qr) ==
            cudaSuccess &&
        qr == cudaDriverEntryPointSuccess)
      return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    return nullptr;
  }();
  return fn;
}

}  // namespace

static bool kv8_encode(CUtensorMap* m, const void* ptr, const cuuint64_t* dims, const cuuint64_t* strides,
                       const cuuint32_t* box) {
  auto fn = kv8_encode_fn();
  const cuuint32_t estr[3] = {1u, 1u, 1u};
  return fn && fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(ptr), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool kv8_map(CUtensorMap* m, const void* ptr, const csa2_kv8_t& c) {
  const cuuint64_t dims[3] = {(cuuint64_t)c.D, kPageRows, (cuuint64_t)c.num_pages * c.H_kv};
  const cuuint64_t strides[2] = {(cuuint64_t)c.D, (cuuint64_t)c.D * kPageRows};
  const cuuint32_t box[3] = {128u, (cuuint32_t)kPageRows, 1u};
  return kv8_encode(m, ptr, dims, strides, box);
}
bool kv8_q_map(CUtensorMap* m, const Kv8AttnArgs& a) {
  const cuuint64_t dims[3] = {256u, (cuuint64_t)a.H, (cuuint64_t)a.b.num_q};
  const cuuint64_t strides[2] = {256u, (cuuint64_t)a.H * 256u};
  const cuuint32_t box[3] = {128u, (cuuint32_t)a.b.G, (cuuint32_t)a.b.QT};
  return kv8_encode(m, a.q_split, dims, strides, box);
}

namespace {

// Rows of a job: the least template that holds the batch's mean queries per sequence times the
// heads of a KV head; above 16 the prefill kernel.  The mean is of what the host knows, the rows of
// q and the sequences, spare and idle ones included.  64 sequences of 8,192 keys, 4 KV heads: 8 rows
// 100 us here, 16 rows 138 (prefill kernel: 222), 32 rows 360 when there was a template for them
// (prefill kernel: 224).
int kv8_rows(int num_q, int num_seqs, int G) {
  const int64_t rows = ((int64_t)num_q + num_seqs - 1) / num_seqs * G;
  return rows <= 8 ? 8 : rows <= 16 ? 16 : kPrefillRows;
}

int kv8_sms() {
  const int n = csa2_device_sms();
  return n > 0 ? n : 148;
}
int kv8_ctas(int R) {
  const int n = kv8_sms() * kv8_ctas_per_sm(R);
  return n < kMaxCtas ? n : kMaxCtas;
}

template <int R, int kUnits>
cudaError_t decode_launch(const csa2_kv8_t& c, const Kv8AttnArgs& a, int ctas, cudaStream_t st) {
  using G = DecGeo<R, kUnits>;
  CUtensorMap tk, tv;
  if (!kv8_map(&tk, c.k, c) || !kv8_map(&tv, c.v, c)) return checked(cudaErrorInvalidValue);
  auto* kernel = kv8_decode_kernel<R, kUnits>;
  cudaError_t e = checked(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)G::kSmem));
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(ctas), dim3(G::kThreads), (size_t)G::kSmem, st, tk, tv, a);
}

}  // namespace
}  // namespace csa2

extern "C" size_t csa2_kv8_attn_workspace(int32_t num_q, int32_t num_seqs, int32_t H, int32_t H_kv,
                                          int32_t D) {
  using namespace csa2;
  if (num_q < 1 || num_seqs < 1 || H < 1 || H_kv < 1 || H % H_kv || H / H_kv > 64 || D < 1)
    return CSA2_STATUS_BYTES;
  const int R = kv8_rows(num_q, num_seqs, H / H_kv), ctas = kv8_ctas(R);
  return CSA2_STATUS_BYTES + up256((size_t)ctas * sizeof(Kv8Desc)) +
         up256((size_t)ctas * 2 * R * sizeof(float2)) + (size_t)ctas * 2 * R * 128 * sizeof(float) +
         (R == kPrefillRows ? up256((size_t)num_q * H * 256) + (size_t)num_q * H * sizeof(float) : 0);
}

extern "C" csa2_status_t csa2_kv8_attn(const uint16_t* q, int64_t q_stride, int32_t num_q, int32_t H,
                                       csa2_kv8_t cache, csa2_seqs_t seqs, const int32_t* q_start,
                                       int32_t window, float softmax_scale, uint16_t* out,
                                       float* lse, void* workspace, size_t ws_bytes, void* stream) {
  using namespace csa2;
  if (num_q < 0 || H < 1 || seqs.num_seqs < 1 || window < 0 ||
      !(softmax_scale > 0.0f && softmax_scale < INFINITY))
    return CSA2_ERR_INVALID_ARG;
  const csa2_status_t bad = kv8_check(cache);
  if (bad != CSA2_OK) return bad;
  if (H % cache.H_kv) return CSA2_ERR_INVALID_ARG;
  const int G = H / cache.H_kv;
  if (G > 64 || num_q > (1 << 28) || seqs.max_pages >= (1 << 24)) return CSA2_ERR_UNSUPPORTED;
  if (q_stride < (int64_t)H * cache.D || q_stride % 8) return CSA2_ERR_INVALID_ARG;
  if (!q_start && (seqs.q_per_seq < 1 || (int64_t)seqs.num_seqs * seqs.q_per_seq != num_q))
    return CSA2_ERR_INVALID_ARG;
  if (!workspace || ws_bytes < csa2_kv8_attn_workspace(num_q, seqs.num_seqs, H, cache.H_kv, cache.D))
    return CSA2_ERR_CAPACITY;
  if (num_q == 0) return CSA2_OK;
  if (!q || !out || !seqs.seq_len || !seqs.block_table || seqs.max_pages < 1 ||
      ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out)) & 15) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255) || !kv8_pointers_ok(cache))
    return CSA2_ERR_INVALID_ARG;
  if (window >= (int64_t)seqs.max_pages * kPageRows) window = 0;        // no key is that far back
  const int R = kv8_rows(num_q, seqs.num_seqs, G), ctas = kv8_ctas(R);
  Kv8AttnArgs a{};
  a.b = Kv8Batch{num_q, seqs.num_seqs, seqs.q_per_seq, seqs.max_pages, window, cache.H_kv, G, R / G,
                 seqs.seq_len, q_start, seqs.block_table};
  a.q = q;
  a.q_stride = q_stride;
  a.H = H;
  a.D = cache.D;
  a.num_pages = cache.num_pages;
  a.k_exp = cache.k_exp;
  a.v_exp = cache.v_exp;
  a.scale_log2 = softmax_scale * 1.4426950408889634f;
  a.out = out;
  a.lse = lse;
  uint8_t* at = static_cast<uint8_t*>(workspace) + CSA2_STATUS_BYTES;
  a.desc = reinterpret_cast<Kv8Desc*>(at);
  at += up256((size_t)ctas * sizeof(Kv8Desc));
  a.part_ml = reinterpret_cast<float2*>(at);
  at += up256((size_t)ctas * 2 * R * sizeof(float2));
  a.part_o = reinterpret_cast<float*>(at);
  at += (size_t)ctas * 2 * R * 128 * sizeof(float);
  if (R == kPrefillRows) {
    a.q_split = at;
    a.q_factor = reinterpret_cast<float*>(at + up256((size_t)num_q * H * 256));
  }
  a.status = static_cast<int*>(workspace);
  a.wait_ns = wait_limit_ns();
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e = R == 8    ? decode_launch<8, 3>(cache, a, ctas, st)
                  : R == 16 ? decode_launch<16, 5>(cache, a, ctas, st)
                            : kv8_prefill_launch(cache, a, ctas, st);
  if (e == cudaSuccess) {
    auto* merge = R == kPrefillRows ? kv8_merge_kernel<1> : kv8_merge_kernel<8>;
    e = launch_pdl(merge, dim3(ctas, R == kPrefillRows ? kMergeBlocks : R),
                   dim3(kMergeWarps * 32), 0, st, R, ctas, (int)H, G, (int)cache.D,
                   (const Kv8Desc*)a.desc, (const float*)a.part_o, (const float2*)a.part_ml, out, lse);
  }
  return e == cudaSuccess ? CSA2_OK : CSA2_ERR_CUDA;
}
