// Rotary positions: out = x with the rotated channels of every head turned by the row's
// position.  Bound by HBM: one read and one write of x.
//
// A row's angles are the same for all its heads, so a CTA first computes the (cos, sin) of its
// rows' pairs into shared memory (one fp64 product and one sincospi each) and then streams the
// heads past them in 16-byte accesses.  A CTA takes several short rows or a slice of a long
// one's heads, so that a single row of many heads still spreads over the GPU.  4,096 rows of
// 64 x 128 bf16 take 27.7 us (4.84 TB/s), 64 decode rows 4.0 us.
#include <cuda_bf16.h>

#include <cfloat>
#include <cmath>

#include "rope.cuh"

namespace csa2 {

csa2_status_t rope_args(const csa2_rope_t* r, RopeArgs* a) {
  double f[kMaxRot / 2];
  const csa2_status_t st = csa2_rope_frequencies(r, f);
  if (st != CSA2_OK) return st;
  a->rot = r->rot_dim;
  a->offset = r->offset;
  a->interleaved = r->interleaved;
  a->amplitude = (float)r->amplitude;
  for (int i = 0; i < r->rot_dim / 2; ++i) a->turns[i] = f[i] / 6.283185307179586476925;
  return CSA2_OK;
}

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeItems = 2048;       // most items (vectors or pairs) wanted per CTA
constexpr int kRopeBatch = 2;          // items of a thread that are loaded before the first is used
constexpr int kRopeTable = 2048;       // (cos, sin) pairs per CTA: 16 KB

struct RopeCall {
  const void* x;
  int64_t x_stride;
  void* out;
  int64_t out_stride;
  int rows, heads, D;
  int rows_per_cta, heads_per_cta;
  const int64_t* pos;
  float sign;                          // -1: the inverse
  RopeArgs r;
};

template <typename T, int V>
struct RopeVec;
template <>
struct RopeVec<float, 4> {
  float v[4];
  __device__ __forceinline__ void set(const uint4& t) {
    v[0] = __uint_as_float(t.x); v[1] = __uint_as_float(t.y);
    v[2] = __uint_as_float(t.z); v[3] = __uint_as_float(t.w);
  }
  __device__ __forceinline__ uint4 get() const {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  }
};
template <>
struct RopeVec<__nv_bfloat16, 8> {
  float v[8];
  __device__ __forceinline__ void set(const uint4& t) {
    const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  __device__ __forceinline__ uint4 get() const {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

__device__ __forceinline__ float rope_in(const float* p) { return *p; }
__device__ __forceinline__ float rope_in(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void rope_out(float* p, float v) { *p = v; }
__device__ __forceinline__ void rope_out(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// kMode 0: any layout, one pair (or one copied channel) per item; 1: interleaved, one vector
// per item; 2: two halves, one vector of each half (or one copied vector) per item
template <typename T, int kMode>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeCall a) {
  constexpr int V = 16 / sizeof(T);
  __shared__ __align__(16) float2 table[kRopeTable];
  pdl_trigger();
  pdl_wait();
  const int rot = a.r.rot, half = rot / 2, off = a.r.offset;
  const int row0 = blockIdx.x * a.rows_per_cta, h0 = blockIdx.y * a.heads_per_cta;
  const int nr = min(a.rows_per_cta, a.rows - row0), nh = min(a.heads_per_cta, a.heads - h0);
  for (int k = threadIdx.x; k < nr * half; k += kRopeThreads) {
    const int r = k / half, i = k - r * half;
    float2 t = rope_turn(a.r, (double)__ldg(a.pos + row0 + r), i);
    t.y *= a.sign;
    table[k] = t;
  }
  __syncthreads();
  const bool copies = a.x != a.out;
  const int turned = kMode == 0 ? half : kMode == 1 ? a.D / V : half / V;
  const int rest = kMode == 1 || !copies ? 0 : kMode == 0 ? a.D - rot : (a.D - rot) / V;
  const int per_head = turned + rest;
  const int n = nr * nh * per_head;
  const uint32_t by_head = 0xFFFFFFFFu / (uint32_t)per_head + 1, by_row = 0xFFFFFFFFu / (uint32_t)nh + 1;
  // x / d for x below 2^16 (d = 1 has no such multiplier)
  auto over = [](uint32_t x, uint32_t mul, int d) { return d == 1 ? (int)x : (int)__umulhi(x, mul); };
  struct Item {
    const T* x;
    T* y;
    const float2* t;
    int j;
  };
  auto item = [&](int k) {
    Item it;
    const int rh = over(k, by_head, per_head);
    it.j = k - rh * per_head;
    const int r = over(rh, by_row, nh), h = h0 + rh - r * nh;
    it.x = static_cast<const T*>(a.x) + (row0 + r) * a.x_stride + (int64_t)h * a.D;
    it.y = static_cast<T*>(a.out) + (row0 + r) * a.out_stride + (int64_t)h * a.D;
    it.t = table + r * half;
    return it;
  };
  if constexpr (kMode != 0) {
    // where the vectors of item j start, and whether they turn
    auto spots = [&](int j, int* ea, int* eb) -> bool {
      if constexpr (kMode == 1) {
        *ea = *eb = j * V;
        return j * V + V > off && j * V < off + rot;
      } else {
        if (j < turned) {
          *ea = off + j * V;
          *eb = *ea + half;
          return true;
        }
        *ea = (j - turned) * V;
        if (*ea >= off) *ea += rot;
        *eb = *ea;
        return false;
      }
    };
    for (int k0 = threadIdx.x; k0 < n; k0 += kRopeBatch * kRopeThreads) {
      uint4 ra[kRopeBatch], rb[kRopeBatch];
#pragma unroll
      for (int b = 0; b < kRopeBatch; ++b) {
        const int k = k0 + b * kRopeThreads;
        if (k < n) {
          const Item it = item(k);
          int ea, eb;
          const bool turns = spots(it.j, &ea, &eb);
          if (turns || copies) ra[b] = *reinterpret_cast<const uint4*>(it.x + ea);
          if (kMode == 2 && turns) rb[b] = *reinterpret_cast<const uint4*>(it.x + eb);
        }
      }
#pragma unroll
      for (int b = 0; b < kRopeBatch; ++b) {
        const int k = k0 + b * kRopeThreads;
        if (k >= n) break;
        const Item it = item(k);
        int ea, eb;
        const bool turns = spots(it.j, &ea, &eb);
        if (!turns) {
          if (copies) *reinterpret_cast<uint4*>(it.y + ea) = ra[b];
          continue;
        }
        RopeVec<T, V> va, vb;
        va.set(ra[b]);
        if constexpr (kMode == 1) {
#pragma unroll
          for (int p = 0; p < V / 2; ++p) {
            const int e = ea + 2 * p, i = (e - off) / 2;
            if (e < off || i >= half) continue;
            const float xa = va.v[2 * p], xb = va.v[2 * p + 1];
            va.v[2 * p] = xa * it.t[i].x - xb * it.t[i].y;
            va.v[2 * p + 1] = xb * it.t[i].x + xa * it.t[i].y;
          }
        } else {
          vb.set(rb[b]);
#pragma unroll
          for (int p = 0; p < V; ++p) {
            const float2 cs = it.t[ea - off + p];
            const float xa = va.v[p], xb = vb.v[p];
            va.v[p] = xa * cs.x - xb * cs.y;
            vb.v[p] = xb * cs.x + xa * cs.y;
          }
          *reinterpret_cast<uint4*>(it.y + eb) = vb.get();
        }
        *reinterpret_cast<uint4*>(it.y + ea) = va.get();
      }
    }
  } else {
    for (int k = threadIdx.x; k < n; k += kRopeThreads) {
      const Item it = item(k);
      if (it.j < half) {
        const int ea = off + (a.r.interleaved ? 2 * it.j : it.j);
        const int eb = ea + (a.r.interleaved ? 1 : half);
        const float xa = rope_in(it.x + ea), xb = rope_in(it.x + eb);
        rope_out(it.y + ea, xa * it.t[it.j].x - xb * it.t[it.j].y);
        rope_out(it.y + eb, xb * it.t[it.j].x + xa * it.t[it.j].y);
      } else {
        int e = it.j - half;
        if (e >= off) e += rot;
        it.y[e] = it.x[e];
      }
    }
  }
}

template <typename T>
cudaError_t rope_launch(RopeCall& a, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  const bool wide = a.D % V == 0 && a.x_stride % V == 0 && a.out_stride % V == 0 &&
                    !((reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.out)) & 15);
  const int mode = !wide ? 0
                   : a.r.interleaved ? 1
                   : (a.r.offset % V == 0 && (a.r.rot / 2) % V == 0) ? 2 : 0;
  const int half = a.r.rot / 2;
  const int per_head = mode == 0 ? a.D - half : mode == 1 ? a.D / V : (a.D - half) / V;
  const int64_t per_row = (int64_t)per_head * a.heads;
  // CTAs for eight per SM before they grow to kRopeItems (registers let 4 to 8 run at a time, 4 of
  // the bf16 form in two halves)
  const int sms = csa2_device_sms() > 0 ? csa2_device_sms() : 148;
  const int64_t even = per_row * a.rows / (8 * sms);
  const int items = even < kRopeThreads ? kRopeThreads : even > kRopeItems ? kRopeItems : (int)even;
  if (per_row >= items) {
    a.rows_per_cta = 1;
    a.heads_per_cta = max(1, items / per_head);
  } else {
    a.heads_per_cta = a.heads;
    a.rows_per_cta = max(1, min((int)(items / per_row), kRopeTable / half));
  }
  const dim3 grid((a.rows + a.rows_per_cta - 1) / a.rows_per_cta,
                  (a.heads + a.heads_per_cta - 1) / a.heads_per_cta);
  auto* kernel = mode == 0 ? rope_kernel<T, 0> : mode == 1 ? rope_kernel<T, 1> : rope_kernel<T, 2>;
  return launch_pdl(kernel, grid, dim3(kRopeThreads), 0, st, a);
}

}  // namespace
}  // namespace csa2

extern "C" csa2_status_t csa2_rope_frequencies(const csa2_rope_t* r, double* freq) {
  if (!r || !freq) return CSA2_ERR_INVALID_ARG;
  if (r->rot_dim < 2 || r->rot_dim > csa2::kMaxRot || r->rot_dim % 2 || r->offset < 0 ||
      r->offset % 2 || (r->interleaved != 0 && r->interleaved != 1) ||
      r->scaling < CSA2_ROPE_NONE || r->scaling > CSA2_ROPE_PARTS)
    return CSA2_ERR_INVALID_ARG;
  // written so that a NaN fails them
  if (!(r->theta > 1.0 && r->theta < 1e30)) return CSA2_ERR_INVALID_ARG;
  if (!(r->amplitude >= FLT_MIN && r->amplitude < 1e6)) return CSA2_ERR_INVALID_ARG;   // fp32 keeps its bits
  if (r->scaling != CSA2_ROPE_NONE && !(r->factor >= 1.0 && r->factor < 1e6))
    return CSA2_ERR_INVALID_ARG;
  if (r->scaling == CSA2_ROPE_BASE && r->rot_dim == 2) return CSA2_ERR_INVALID_ARG;
  if (r->scaling == CSA2_ROPE_PARTS &&
      !(r->orig_len > 0.0 && r->orig_len < 1e15 && r->slow < r->fast && r->slow >= 0.0 &&
        r->fast < 1e15))
    return CSA2_ERR_INVALID_ARG;
  const double d = r->rot_dim;
  const double theta =
      r->scaling == CSA2_ROPE_BASE ? r->theta * std::pow(r->factor, d / (d - 2.0)) : r->theta;
  for (int i = 0; i < r->rot_dim / 2; ++i) {
    double f = std::pow(theta, -2.0 * i / d);
    if (r->scaling == CSA2_ROPE_LINEAR) f /= r->factor;
    if (r->scaling == CSA2_ROPE_PARTS) {
      const double turns = r->orig_len * f / 6.283185307179586476925;
      double g = (turns - r->slow) / (r->fast - r->slow);
      g = g < 0.0 ? 0.0 : g > 1.0 ? 1.0 : g;
      f = g * f + (1.0 - g) * f / r->factor;
    }
    freq[i] = f;
  }
  return CSA2_OK;
}

extern "C" csa2_status_t csa2_rope(const void* x, int64_t x_stride, void* out, int64_t out_stride,
                                   int32_t rows, int32_t heads, int32_t D, int32_t dtype,
                                   const int64_t* pos, const csa2_rope_t* rope, int32_t inverse,
                                   void* stream) {
  using namespace csa2;
  if (rows < 0 || heads < 1 || D < 2 || (dtype != 0 && dtype != 1) ||
      (inverse != 0 && inverse != 1))
    return CSA2_ERR_INVALID_ARG;
  if (D > 4096 || D % 2 || heads > 65535 || rows > (1 << 30)) return CSA2_ERR_UNSUPPORTED;
  if (x_stride < (int64_t)heads * D || out_stride < (int64_t)heads * D) return CSA2_ERR_INVALID_ARG;
  RopeCall a{};
  const csa2_status_t bad = rope_args(rope, &a.r);
  if (bad != CSA2_OK) return bad;
  if ((int64_t)a.r.offset + a.r.rot > D) return CSA2_ERR_INVALID_ARG;
  if (rows == 0) return CSA2_OK;
  if (!x || !out || !pos || (x == out && x_stride != out_stride)) return CSA2_ERR_INVALID_ARG;
  const uintptr_t size = dtype == 0 ? 2 : 4;
  if ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(out)) & (size - 1))
    return CSA2_ERR_INVALID_ARG;
  a.x = x;
  a.x_stride = x_stride;
  a.out = out;
  a.out_stride = out_stride;
  a.rows = rows;
  a.heads = heads;
  a.D = D;
  a.pos = pos;
  a.sign = inverse ? -1.0f : 1.0f;
  const cudaError_t e = dtype == 0 ? rope_launch<__nv_bfloat16>(a, (cudaStream_t)stream)
                                   : rope_launch<float>(a, (cudaStream_t)stream);
  return e == cudaSuccess ? CSA2_OK : CSA2_ERR_CUDA;
}
