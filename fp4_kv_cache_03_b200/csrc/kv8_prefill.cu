// Causal attention over the paged 8-bit cache, for many query rows per KV head (prefill).
//
// What it cannot do without are the tensor cores and, as much, the exponentials: a 128 x 128 tile of
// S costs 1,024 cycles of MMAs (below) and 1,024 of the SM's 16 ex2 per cycle.
//
// A job is 256 rows (queries x the G heads of one KV head) in two halves of 128, each with a
// softmax warpgroup of one thread per row, so that neither maximum nor sum crosses threads.
//   S[row, key] = Q . K^T   K's codes straight from TMA as E4M3; Q (bf16) as two E4M3 terms
//                           hi + lo: 2 x K = 32 steps at FP8 rate, the cost of one bf16
//                           product, with no conversion of K.  A kernel ahead splits all of Q
//                           into the workspace, and a job's rows come by two TMA boxes (split by
//                           the softmax warps at each job's start it cost them 8,000 cycles)
//   O[row, d] += P . V      P in f16 (11 bits, down to 2^-28 of the reference's weight),
//                           written over S in tensor memory; V's codes widened to f16 (exact)
//                           by four warps, once per tile for both halves
// P has 128 x 128 values per tile, V 128 x D for twice as many products: splitting P into E4M3
// terms as the decode kernel does would cost three conversions per value here.
// S and P go in two parts of 64 keys: while one part is weighed, the MMAs of the other part and of
// the other half run.  S of a part's next tile is issued right behind its P . V, which reads P from
// the columns that S overwrites; MMAs of one thread run in order.  Scales as in the decode kernel:
// 2^ek multiplies S, ev is added to the exponent, the sum takes w * 2^-ev.  A row's reference moves
// only when weights come near f16's largest: O is rescaled then, by the row's own warp.
//
// 2,048 queries over 10,240 tokens, 64 heads on 8 of 128: 718 to 727 us, 861 to 850 TFLOP/s; the
// tensor pipe and the exponential unit are both 40% busy, and what bounds it are the softmax warps'
// latencies (2 such warps per scheduler).
#include <cuda.h>

#include "kv8_attn.cuh"

namespace csa2 {
namespace {

constexpr int kPfThreads = 512;               // 8 softmax warps, 4 converters, producer, issuer, 2 idle
constexpr int kKStages = 3, kVStages = 2, kHBufs = 2;
constexpr float kPfTop = 3.0f;                // a fresh reference's weight is 2^3 ...
constexpr float kPfSum = 65000.0f;            // ... and 16 neighbouring ones sum to no more than this
constexpr float kPfRaise = 10.0f;             // log2 of a weight that is taken to 2^3 when they do

constexpr uint32_t kOffQ = 0;                 // [hi, lo][256 rows][128 B]
constexpr uint32_t kOffK = kOffQ + 4 * kUnit;
constexpr uint32_t kOffV = kOffK + kKStages * kUnit;
constexpr uint32_t kOffH = kOffV + kVStages * kUnit;      // f16 V: [64-channel chunk][128 keys][128 B]
constexpr uint32_t kHBytes = 2 * kUnit;
constexpr uint32_t kPfSmem = 1024 + kOffH + kHBufs * kHBytes;

struct PfInfo {
  float kf[8], ve[8], vinv[8];
  int ok;
};

struct PfSmem {
  uint64_t k_full[kKStages], k_empty[kKStages], v_full[kVStages], v_empty[kVStages];
  uint64_t h_full[kHBufs], h_empty[kHBufs], info_full[kInfo];
  uint64_t q_full, q_empty, s_full[2][2], p_full[2][2], o_done[2][2], drain;   // [half][part]
  int64_t red64[kPfThreads / 32];
  Kv8Share share;
  uint32_t tmem_base;
  int abort;
  alignas(16) PfInfo info[kInfo];
};

// One half of a job: its rows, their positions, and the key tiles (absolute) that any sees.
struct Half {
  int rows, p_first, p_last, lo, hi;
};
__device__ __forceinline__ Half half_of(const Kv8Batch& b, const Kv8Walk& w, int x) {
  Half r;
  const int all = w.tile.nq * b.G;
  r.rows = x ? max(0, all - 128) : min(all, 128);
  r.p_first = w.tile.p0 + (x ? 128 / b.G : 0);
  r.p_last = w.tile.p0 + (x ? all - 1 : min(all, 128) - 1) / b.G;
  r.lo = b.window && r.p_first >= b.window ? (r.p_first - b.window + 1) / kPageRows : 0;
  r.hi = r.rows > 0 && r.p_last >= 0 ? r.p_last / kPageRows + 1 : 0;
  // within the share
  r.lo = max(r.lo, w.tile.kt0 + w.kt);
  r.hi = min(r.hi, w.tile.kt0 + w.kt_end);
  return r;
}

// two fp32 in a register pair, and the packed arithmetic on them
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pair(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 both(f32x2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// 64 consecutive columns of the thread's lane as 32 pairs, one wait
__device__ __forceinline__ void tmem_ld64x2(uint32_t taddr, f32x2* v) {
  uint32_t r[2][32];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[i][0]), "=r"(r[i][1]), "=r"(r[i][2]), "=r"(r[i][3]), "=r"(r[i][4]), "=r"(r[i][5]),
          "=r"(r[i][6]), "=r"(r[i][7]), "=r"(r[i][8]), "=r"(r[i][9]), "=r"(r[i][10]),
          "=r"(r[i][11]), "=r"(r[i][12]), "=r"(r[i][13]), "=r"(r[i][14]), "=r"(r[i][15]),
          "=r"(r[i][16]), "=r"(r[i][17]), "=r"(r[i][18]), "=r"(r[i][19]), "=r"(r[i][20]),
          "=r"(r[i][21]), "=r"(r[i][22]), "=r"(r[i][23]), "=r"(r[i][24]), "=r"(r[i][25]),
          "=r"(r[i][26]), "=r"(r[i][27]), "=r"(r[i][28]), "=r"(r[i][29]), "=r"(r[i][30]),
          "=r"(r[i][31])
        : "r"(taddr + i * 32));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 2; ++i)                 // no use moves above the wait
    asm volatile(""
                 : "+r"(r[i][0]), "+r"(r[i][1]), "+r"(r[i][2]), "+r"(r[i][3]), "+r"(r[i][4]),
                   "+r"(r[i][5]), "+r"(r[i][6]), "+r"(r[i][7]), "+r"(r[i][8]), "+r"(r[i][9]),
                   "+r"(r[i][10]), "+r"(r[i][11]), "+r"(r[i][12]), "+r"(r[i][13]), "+r"(r[i][14]),
                   "+r"(r[i][15]), "+r"(r[i][16]), "+r"(r[i][17]), "+r"(r[i][18]), "+r"(r[i][19]),
                   "+r"(r[i][20]), "+r"(r[i][21]), "+r"(r[i][22]), "+r"(r[i][23]), "+r"(r[i][24]),
                   "+r"(r[i][25]), "+r"(r[i][26]), "+r"(r[i][27]), "+r"(r[i][28]), "+r"(r[i][29]),
                   "+r"(r[i][30]), "+r"(r[i][31])
                 :
                 : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i)
    v[i] = pair(__uint_as_float(r[i >> 4][2 * i & 31]), __uint_as_float(r[i >> 4][(2 * i & 31) + 1]));
}
__device__ __forceinline__ void tmem_st32u(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31])
      : "memory");
}
// kind::f16 with f16 A and B (format 0), fp32 D, B MN-major
constexpr uint32_t idesc_f16_bmn(int M, int N) {
  return (1u << 4) | (1u << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__global__ void __launch_bounds__(kPfThreads, 1)
    kv8_prefill_kernel(const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v,
                       const __grid_constant__ CUtensorMap tm_q, const Kv8AttnArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ PfSmem sm;
  uint8_t* base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort = &sm.abort;
  constexpr int kConvert = 8, kProducer = 12, kIssuer = 13;

  if (tid == 0) {
    for (int i = 0; i < kKStages; ++i) { mbar_init(&sm.k_full[i], 1); mbar_init(&sm.k_empty[i], 1); }
    for (int i = 0; i < kVStages; ++i) { mbar_init(&sm.v_full[i], 1); mbar_init(&sm.v_empty[i], 4); }
    for (int i = 0; i < kHBufs; ++i) { mbar_init(&sm.h_full[i], 4); mbar_init(&sm.h_empty[i], 1); }
    for (int i = 0; i < kInfo; ++i) mbar_init(&sm.info_full[i], 1);
    for (int i = 0; i < 2; ++i) {
      for (int p = 0; p < 2; ++p) {
        mbar_init(&sm.s_full[i][p], 1);
        mbar_init(&sm.p_full[i][p], 4);
        mbar_init(&sm.o_done[i][p], 1);
      }
    }
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_empty, 1);
    mbar_init(&sm.drain, 1);
    sm.abort = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    tma_prefetch_desc(&tm_q);
  }
  if (warp == kIssuer) { tmem_alloc(&sm.tmem_base, 512); tmem_relinquish(); }
  pdl_wait();
  kv8_share(a.b, blockIdx.x, gridDim.x, sm.red64, &sm.share, blockIdx.x == 0 ? a.status : nullptr);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();                               // after the allocation, as in the decode kernel
  const uint32_t tmem = sm.tmem_base;          // S0, S1 (P over them), O0, O1: 128 columns each
  const int T = (int)(sm.share.end - sm.share.begin);
  Kv8Walk w;
  if (T > 0) w.start(a.b, sm.share);

  // The softmax warps hold a row of S: 192 registers for them, 64 for the others (the sum is what
  // 512 threads of 128 were launched with).
  if (warp == kProducer) {
    // ------------------------------ pages -> K and V stages ------------------------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    int kb = 0, at = w.kt, z = -1;
    bool fresh = true, ok = true;
    uint2 kx = make_uint2(0, 0), vx = kx;
    int done_k = 0, done_v = 0, done_q = 0;    // tiles, and jobs' Q, whose loads were issued
    for (int g = 0; g < T; ++g) {
      if (!fresh && at == w.kt_end) {
        w.next(a.b);
        at = w.kt;
        fresh = true;
      }
      if (fresh || at - kb == 32) {            // the lanes fetch 32 tiles' pages and scales
        kb = at;
        fresh = false;
        z = -1;
        const int t = at + lane;
        if (t < w.kt_end && w.tile.p0 + w.tile.nq > 0) {
          const int page = __ldg(a.b.block_table + (int64_t)w.s * a.b.max_pages + w.tile.kt0 + t);
          if (page < 0 || page >= a.num_pages) {
            report(a.status, CSA2_ERR_CAPACITY);
          } else {
            z = page * a.b.H_kv + w.h;
            kx = __ldg(reinterpret_cast<const uint2*>(a.k_exp) + z);
            vx = __ldg(reinterpret_cast<const uint2*>(a.v_exp) + z);
          }
        }
      }
      const int src = at - kb;
      const int row = __shfl_sync(0xffffffffu, z, src);
      const uint32_t k0 = __shfl_sync(0xffffffffu, kx.x, src), k1 = __shfl_sync(0xffffffffu, kx.y, src);
      const uint32_t v0 = __shfl_sync(0xffffffffu, vx.x, src), v1 = __shfl_sync(0xffffffffu, vx.y, src);
      PfInfo& inf = sm.info[g % kInfo];
      if (lane < 8) inf.kf[lane] = exp2i(kv8_exp((lane < 4 ? k0 : k1) >> (8 * (lane & 3)) & 255u));
      else if (lane < 16) inf.ve[lane - 8] = 8.0f + (float)kv8_exp((lane < 12 ? v0 : v1) >> (8 * (lane & 3)) & 255u);
      else if (lane < 24) inf.vinv[lane - 16] = exp2i(-8 - kv8_exp((lane < 20 ? v0 : v1) >> (8 * (lane & 3)) & 255u));
      else if (lane == 24) inf.ok = row >= 0;
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sm.info_full[g % kInfo]);
        const int ks = g % kKStages, vs = g % kVStages;
        if (at == w.kt) {                      // the job's Q, when the job before is done with its own
          ok = kv8_wait(&sm.q_empty, (uint32_t)done_q & 1u ^ 1u, abort, a.status, a.wait_ns);
          if (ok) {
            mbar_arrive_expect_tx(&sm.q_full, 2 * 128 * a.b.QT * a.b.G);
            for (int k = 0; k < 2; ++k)
              tma_load_3d(base + kOffQ + k * 2 * kUnit, &tm_q, k * 128, w.h * a.b.G,
                          w.seq.q0 + w.i * a.b.QT, &sm.q_full);
            ++done_q;
          }
        }
        ok = ok && kv8_wait(&sm.k_empty[ks], (uint32_t)(g / kKStages) & 1u ^ 1u, abort, a.status, a.wait_ns);
        if (ok) {
          if (row >= 0) {
            mbar_arrive_expect_tx(&sm.k_full[ks], kUnit);
            tma_load_3d(base + kOffK + ks * kUnit, &tm_k, 0, 0, row, &sm.k_full[ks]);
          } else {
            mbar_arrive(&sm.k_full[ks]);
          }
          done_k = g + 1;
          ok = kv8_wait(&sm.v_empty[vs], (uint32_t)(g / kVStages) & 1u ^ 1u, abort, a.status, a.wait_ns);
        }
        if (ok) {
          if (row >= 0) {
            mbar_arrive_expect_tx(&sm.v_full[vs], kUnit);
            tma_load_3d(base + kOffV + vs * kUnit, &tm_v, 0, 0, row, &sm.v_full[vs]);
          } else {
            mbar_arrive(&sm.v_full[vs]);
          }
          done_v = g + 1;
        }
      }
      ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
      if (!ok) break;
      ++at;
    }
    // no load of this CTA may still be landing when it exits
    if (lane == 0) {
      if (done_q > 0) mbar_drain(&sm.q_full, (uint32_t)(done_q - 1) & 1u);
      for (int g = max(0, done_k - kKStages); g < done_k; ++g)
        mbar_drain(&sm.k_full[g % kKStages], (uint32_t)(g / kKStages) & 1u);
      for (int g = max(0, done_v - kVStages); g < done_v; ++g)
        mbar_drain(&sm.v_full[g % kVStages], (uint32_t)(g / kVStages) & 1u);
    }
  } else if (warp == kIssuer) {
    // ------------------------------ MMAs ------------------------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (T > 0) {
      const uint32_t leader = elect_one();
      const uint32_t id_s = idesc_e4m3(128, 64), id_o = idesc_f16_bmn(128, a.D);
      const int ksteps = (a.D + 31) / 32;
      // descriptors; the address field counts 16 bytes
      const uint64_t sq0 = sdesc_sw128(smem_u32(base + kOffQ), 16, 1024);
      const uint64_t sk0 = sdesc_sw128(smem_u32(base + kOffK), 16, 1024);
      const uint64_t sh0 = sdesc_sw128(smem_u32(base + kOffH), kUnit, 1024);
      int at = w.kt;
      uint32_t np[2] = {0, 0}, job = 0;         // P so far of each half; jobs
      bool pend[2] = {false, false}, fresh_o[2] = {false, false};
      bool ok = true;
      Half half[2] = {half_of(a.b, w, 0), half_of(a.b, w, 1)};
      auto wait = [&](uint64_t* b, uint32_t parity) {
        ok = ok && kv8_wait_warp(b, parity & 1u, abort, a.status, a.wait_ns);
      };
      for (int t = 0; t <= T && ok; ++t) {
        const int ks = t % kKStages, hb = (t - 1) & 1;
        int kt = 0;
        if (t < T) {
          if (at == w.kt_end) {
            w.next(a.b);
            at = w.kt;
            half[0] = half_of(a.b, w, 0);
            half[1] = half_of(a.b, w, 1);
          }
          kt = w.tile.kt0 + at;
          if (at == w.kt) wait(&sm.q_full, job++);
          ++at;
          wait(&sm.k_full[ks], t / kKStages);
        }
        if (t > 0) wait(&sm.h_full[hb], (t - 1) / kHBufs);
        const bool act[2] = {t < T && kt >= half[0].lo && kt < half[0].hi,
                             t < T && kt >= half[1].lo && kt < half[1].hi};
        bool first[2];
#pragma unroll 1
        for (int part = 0; part < 2; ++part) {
          const uint64_t vd = sh0 + (uint32_t)(hb * (kHBytes >> 4) + part * 512);   // 64 keys: 8 KB
          const uint64_t kd = sk0 + (uint32_t)(ks * (kUnit >> 4) + part * 512);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint32_t t_s = tmem + x * 128 + part * 64;
            if (pend[x]) {                     // P . V of tile t - 1
              wait(&sm.p_full[x][part], np[x]);
              if (ok) {
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < 4; ++k)    // 16 keys, 2048 bytes each
                  warp_umma_f16_ta(leader, tmem + 256 + x * 128, t_s + k * 8, vd + k * 128, id_o,
                                   part > 0 || k > 0 || !fresh_o[x]);
                warp_commit(leader, &sm.o_done[x][part]);
              }
            }
            if (act[x]) {
              first[x] = kt == half[x].lo;
              if (ok) {
                tc_fence_after();
                const uint64_t ad = sq0 + x * (kUnit >> 4);
#pragma unroll
                for (int k = 0; k < 4; ++k)    // 32 channels, 32 bytes each
                  if (k < ksteps) {
                    warp_umma_e4m3(leader, t_s, ad + k * 2, kd + k * 2, id_s, k > 0);
                    warp_umma_e4m3(leader, t_s, ad + 2 * (kUnit >> 4) + k * 2, kd + k * 2, id_s, 1);
                  }
                warp_commit(leader, &sm.s_full[x][part]);
              }
            }
          }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (pend[x]) ++np[x];
          pend[x] = act[x];
          if (act[x]) fresh_o[x] = first[x];
        }
        if (!ok) break;
        if (t < T) warp_commit(leader, &sm.k_empty[ks]);
        if (t < T && at == w.kt_end) warp_commit(leader, &sm.q_empty);
        if (t > 0) warp_commit(leader, &sm.h_empty[hb]);
      }
      // every MMA this warp issued has completed before the CTA frees TMEM and exits
      warp_commit(leader, &sm.drain);
      mbar_drain(&sm.drain, 0);
      __syncwarp();
    }
  } else if (warp >= kConvert && warp < kProducer) {
    // ------------------------------ V codes -> f16 ------------------------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    const int j = tid - kConvert * 32;         // its row
    auto wait = [&](uint64_t* b, uint32_t parity) {
      if (lane == 0) kv8_wait(b, parity & 1u, abort, a.status, a.wait_ns);
      __syncwarp();
    };
    int at = w.kt;
    for (int g = 0; g < T; ++g, ++at) {
      if (at == w.kt_end) {
        w.next(a.b);
        at = w.kt;
      }
      const int vs = g % kVStages, hb = g % kHBufs;
      const int keys = w.tile.p0 + w.tile.nq - (w.tile.kt0 + at) * kPageRows;  // seen by any row
      wait(&sm.info_full[g % kInfo], g / kInfo);
      const bool loaded = sm.info[g % kInfo].ok != 0;
      wait(&sm.v_full[vs], g / kVStages);
      wait(&sm.h_empty[hb], g / kHBufs + 1);
      uint8_t* src = base + kOffV + vs * kUnit;
      uint8_t* dst = base + kOffH + hb * kHBytes;
      // Rows behind the last key, or of a page that is not there, may hold NaN codes: zeros.  A code
      // seeemmm shifted into place is an f16 of 2^-8 its value (subnormals too): the softmax
      // takes the 2^8 along with the scale.
      const bool keep = loaded && j < keys;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if (half * 64 >= a.D) break;
        uint4 v[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) v[c] = *reinterpret_cast<const uint4*>(src + sw128(j, half * 64 + c * 16));
        uint8_t* d = dst + half * kUnit;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t in[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
          uint32_t o[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint32_t x = __byte_perm(keep ? in[k >> 1] : 0u, 0u, k & 1 ? 0x3424u : 0x1404u);
            o[k] = (x & 0x80008000u) | (x & 0x7F007F00u) >> 1;
          }
          *reinterpret_cast<uint4*>(d + sw128(j, c * 32)) = make_uint4(o[0], o[1], o[2], o[3]);
          *reinterpret_cast<uint4*>(d + sw128(j, c * 32 + 16)) = make_uint4(o[4], o[5], o[6], o[7]);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sm.v_empty[vs]);
        mbar_arrive(&sm.h_full[hb]);
      }
    }
  } else if (warp > kIssuer) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
  } else {
    // ------------------------------ softmax: one row per thread ------------------------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
    const int x = warp >> 2, quad = warp & 3, row = quad * 32 + lane;
    const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
    const uint32_t t_s = tmem + lane_base + x * 128, t_o = tmem + lane_base + 256 + x * 128;
    auto wait = [&](uint64_t* b, uint32_t parity) {
      if (!mbar_try_wait(b, parity & 1u)) kv8_wait(b, parity & 1u, abort, a.status, a.wait_ns);
      __syncwarp();
    };
    // softmax_scale * log2(e) * 2^e of the thread's row of Q in the walker's job
    auto row_factor = [&](const Half& hf) {
      const int r = x * 128 + row;
      return row < hf.rows ? __ldg(a.q_factor + (int64_t)(w.seq.q0 + w.i * a.b.QT + r / a.b.G) * a.H +
                                   w.h * a.b.G + r % a.b.G)
                           : 0.0f;
    };
    Half hf{0, 0, 0, 0, 0};
    float factor = 0.0f;
    if (T > 0) {
      hf = half_of(a.b, w, x);
      factor = row_factor(hf);
    }
    int g0 = 0;                                // the share's tiles before the job
    uint32_t n = 0;                            // tiles of this half so far
    bool sat_out = false;                      // it saw nothing of the job before
    Kv8Desc d{0, 0, 0, 0, 0};
    while (!w.done()) {
      if (!w.begins()) d.head_ends = w.ends();
      if (w.begins() && !w.ends())
        d = Kv8Desc{1, d.head_ends, w.seq.q0 + w.i * a.b.QT, w.tile.nq * a.b.G, w.h};
      const int t_row = row < hf.rows ? w.tile.p0 + (x * 128 + row) / a.b.G : -1;
      // a thread without a row weighs everything 0
      float ref = row < hf.rows ? 0.0f : 1e30f, sum = 0.0f;
      bool have = row >= hf.rows;              // ref comes from a weight of the row
      // A parity tells neighbouring rounds of the ring of scales apart, no more, and a half that saw
      // nothing of the jobs before (few rows, positions before the first token) may be rounds
      // ahead of the producer.  S of its first tile comes after that tile's scales were written,
      // and nobody overwrites those before this half's P is there.  (Between two jobs that it
      // sees, a half sits out three tiles at most, and the parity does.)
      if (sat_out && hf.lo < hf.hi) wait(&sm.s_full[x][0], n);
      sat_out = hf.lo >= hf.hi;
      for (int kt = hf.lo; kt < hf.hi; ++kt, ++n) {
        const int g = g0 + kt - (w.tile.kt0 + w.kt);
        const int j0 = kt * kPageRows;
        wait(&sm.info_full[g % kInfo], g / kInfo);
        const PfInfo& inf = sm.info[g % kInfo];
        const bool loaded = inf.ok != 0;
        const bool whole = loaded && j0 + kPageRows - 1 <= hf.p_first &&
                           (!a.b.window || j0 > hf.p_last - a.b.window);
        auto multiplier = [&](int b) {         // never 0: the -inf of a masked column has to stay -inf
          const float m = factor * inf.kf[b];
          return m == 0.0f ? 1e-37f : m;
        };
        // two parts of 64 keys: while one is weighed, the MMAs of the other part run
#pragma unroll 1
        for (int part = 0; part < 2; ++part) {
          const uint32_t t_p = t_s + part * 64;
          float mul[4], off[4];
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            mul[b] = multiplier(part * 4 + b);
            off[b] = inf.ve[part * 4 + b];
          }
          wait(&sm.s_full[x][part], n);
          tc_fence_after();
          if (!whole) {                        // columns that the row does not see become -inf
            const int j1 = j0 + part * 64;
            const int hi = loaded ? t_row - j1 : -1, lo = a.b.window ? t_row - a.b.window - j1 : -1;
#pragma unroll 1
            for (int c0 = 0; c0 < 64; c0 += 32) {
              float v[32];
              tmem_ld32(t_p + c0, t_p + c0 + 16, v);
#pragma unroll
              for (int c = 0; c < 32; ++c) v[c] = c0 + c <= hi && c0 + c > lo ? v[c] : -INFINITY;
              tmem_st16(t_p + c0, v);
              tmem_st16(t_p + c0 + 16, v + 16);
            }
            tmem_wait_st();
          }
          // the part's largest exponent
          auto largest = [&]() -> float {
            float m = -INFINITY;
#pragma unroll 1
            for (int b = 0; b < 4; ++b) {
              float v[16];
              tmem_ldn<16>(t_p + b * 16, v);
              const float f = multiplier(part * 4 + b), o = inf.ve[part * 4 + b];
#pragma unroll
              for (int c = 0; c < 16; ++c) m = fmaxf(m, fmaf(v[c], f, o));
            }
            return m;
          };
          if (__any_sync(0xffffffffu, !have)) {  // nothing of O, sum or P depends on ref yet
            const float m = largest();
            if (!have && m > -INFINITY) {
              ref = m - kPfTop;
              have = true;
            }
          }
          // Weights under the reference as f16, their sum, and whether one may be over the limit:
          // 16 of them sum to more than 65,000 only where one is over 2^11.9, so no maximum is needed,
          // and where they do not, none is past f16's 65,504.  A fresh reference's weight of 2^3
          // keeps the small weights of long contexts (2^0 would lose those of 2^-25 of the largest);
          // more would move references too often (2,048-token chunk: 2^0 711 us, 2^3 718, 2^4 722).
          // A part's body is as much as pays to unroll: over the whole tile it outgrows the
          // instruction caches (18% slower), over half a part its latencies show.
          uint32_t p[32];
          float add;
          auto weigh = [&]() -> bool {
            f32x2 s[32];
            tmem_ld64x2(t_p, s);
            float most = 0.0f;
            add = 0.0f;
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              const float o = off[b] - ref;
              const f32x2 m2 = pair(mul[b], mul[b]), o2 = pair(o, o);
              f32x2 both_sums = pair(0.0f, 0.0f);
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                float2 v = both(fma2(s[b * 8 + c], m2, o2));
                v.x = ex2(v.x);
                v.y = ex2(v.y);
                both_sums = add2(both_sums, pair(v.x, v.y));
                const __half2 h = __floats2half2_rn(v.x, v.y);
                p[b * 8 + c] = *reinterpret_cast<const uint32_t*>(&h);
              }
              const float2 v = both(both_sums);
              add = fmaf(v.x + v.y, inf.vinv[part * 4 + b], add);
              most = fmaxf(most, v.x + v.y);
            }
            return most > kPfSum;
          };
#pragma unroll 1
          while (__any_sync(0xffffffffu, weigh())) {
            // rarely: raise the reference, take sum and O along, and weigh the part again
            const float m = largest();
            const float up = m - ref > kPfRaise ? ceilf(m - ref) - kPfTop : 0.0f;
            const float alpha = ex2(-up);
            ref += up;
            sum *= alpha;
            if (kt > hf.lo || part > 0) {
              wait(&sm.o_done[x][part ^ 1], n + part - 1);   // the part before
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < a.D; c += 16) {
                float o[16];
                tmem_ldn<16>(t_o + c, o);
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] *= alpha;
                tmem_st16(t_o + c, o);
              }
              tmem_wait_st();
            }
            if (!__any_sync(0xffffffffu, up > 0.0f)) break;      // infinite weights: as they are
          }
          tmem_st32u(t_p, p);
          sum += add;
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.p_full[x][part]);
        }
      }
      const bool any = hf.lo < hf.hi;
      const bool final = w.begins() && w.ends();
      const int slot = 2 * blockIdx.x + (w.begins() ? 1 : 0), r = x * 128 + row;
      const bool mine = row < hf.rows;
      const int64_t hrow = (int64_t)(w.seq.q0 + w.i * a.b.QT + r / a.b.G) * a.H + w.h * a.b.G + r % a.b.G;
      g0 += w.kt_end - w.kt;
      w.next(a.b);
      if (!w.done()) {
        hf = half_of(a.b, w, x);
        factor = row_factor(hf);
      }
      if (any) {
        wait(&sm.o_done[x][1], n - 1);
        tc_fence_after();
      }
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll 1
      for (int c = 0; c < a.D; c += 16) {
        float o[16];
        if (any) {
          tmem_ldn<16>(t_o + c, o);
        } else {
#pragma unroll
          for (int k = 0; k < 16; ++k) o[k] = 0.0f;
        }
        if (!mine) continue;
        if (final) {
          uint32_t b[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const __nv_bfloat162 two = __floats2bfloat162_rn(o[2 * k] * inv, o[2 * k + 1] * inv);
            b[k] = *reinterpret_cast<const uint32_t*>(&two);
          }
          uint4* dst = reinterpret_cast<uint4*>(a.out + hrow * a.D + c);
          dst[0] = make_uint4(b[0], b[1], b[2], b[3]);
          dst[1] = make_uint4(b[4], b[5], b[6], b[7]);
        } else {
          float4* dst = reinterpret_cast<float4*>(a.part_o + ((int64_t)slot * kPrefillRows + r) * 128 + c);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            dst[k] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
        }
      }
      tc_fence_before();
      if (mine) {
        if (!final)
          a.part_ml[(int64_t)slot * kPrefillRows + r] = make_float2(sum == 0.0f ? -INFINITY : ref, sum);
        else if (a.lse)
          a.lse[hrow] = sum == 0.0f ? -INFINITY : (ref + lg2(sum)) * 0.6931471805599453f;
      }
    }
    if (tid == 0) a.desc[blockIdx.x] = d;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kIssuer) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// All rows of Q as two E4M3 terms, scaled by a power of two so that a row's largest is in (224, 448]:
// 16 lanes of 8 channels per row.  Channels behind D are zeros.
constexpr int kSplitThreads = 256;
__global__ void __launch_bounds__(kSplitThreads) kv8_split_q_kernel(const uint16_t* q, int64_t q_stride,
                                                                    int64_t rows, int H, int D,
                                                                    float scale_log2, uint8_t* split,
                                                                    float* factor) {
  pdl_trigger();
  pdl_wait();
  const int64_t row = ((int64_t)blockIdx.x * kSplitThreads + threadIdx.x) >> 4;
  const int ch = (threadIdx.x & 15) * 8;
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (row < rows && ch < D)
    v = __ldg(reinterpret_cast<const uint4*>(q + row / H * q_stride + row % H * D + ch));
  const uint32_t in[4] = {v.x, v.y, v.z, v.w};
  uint32_t top = __vmaxu2(__vmaxu2(in[0] & 0x7FFF7FFFu, in[1] & 0x7FFF7FFFu),
                          __vmaxu2(in[2] & 0x7FFF7FFFu, in[3] & 0x7FFF7FFFu));
  top = max(top & 0xFFFFu, top >> 16);
#pragma unroll
  for (int d = 8; d; d >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
  if (row >= rows) return;
  const int e = max(-120, min(119, kv8_least_exp(__uint_as_float(top << 16))));
  const float f = exp2i(-e);
  uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float p = __uint_as_float(in[k] << 16) * f, s = __uint_as_float(in[k] & 0xFFFF0000u) * f;
    const uint32_t h2 = e4m3x2(p, s);
    const float2 hv = e4m3x2_value(h2);
    hi[k >> 1] |= h2 << (16 * (k & 1));
    lo[k >> 1] |= e4m3x2(p - hv.x, s - hv.y) << (16 * (k & 1));
  }
  uint8_t* dst = split + row * 256 + ch;
  *reinterpret_cast<uint2*>(dst) = make_uint2(hi[0], hi[1]);
  *reinterpret_cast<uint2*>(dst + 128) = make_uint2(lo[0], lo[1]);
  // a row with an infinity or a NaN gives NaN, not a saturated answer
  if (ch == 0) factor[row] = top >= 0x7F80u ? __int_as_float(0x7FC00000) : scale_log2 * exp2i(e);
}

}  // namespace

cudaError_t kv8_prefill_launch(const csa2_kv8_t& c, const Kv8AttnArgs& a, int ctas, cudaStream_t st) {
  CUtensorMap tk, tv, tq;
  if (!kv8_map(&tk, c.k, c) || !kv8_map(&tv, c.v, c) || !kv8_q_map(&tq, a)) return checked(cudaErrorInvalidValue);
  const int64_t rows = (int64_t)a.b.num_q * a.H, blocks = (rows * 16 + kSplitThreads - 1) / kSplitThreads;
  if (blocks > 0x7FFFFFFF) return checked(cudaErrorInvalidValue);
  const cudaError_t s = launch_pdl(kv8_split_q_kernel, dim3((unsigned)blocks), dim3(kSplitThreads), 0, st, a.q,
                                   a.q_stride, rows, a.H, a.D, a.scale_log2, a.q_split, a.q_factor);
  if (s != cudaSuccess) return s;
  const cudaError_t e = checked(cudaFuncSetAttribute(
      kv8_prefill_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kPfSmem));
  if (e != cudaSuccess) return e;
  return launch_pdl(kv8_prefill_kernel, dim3(ctas), dim3(kPfThreads), (size_t)kPfSmem, st, tk, tv, tq, a);
}

}  // namespace csa2
