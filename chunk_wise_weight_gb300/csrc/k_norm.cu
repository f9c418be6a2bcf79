// k_norm.cu -- layer norm over the last dimension and its gradients.
//
//   y = (x - mu) rstd w + b,  mu = mean(x), rstd = 1 / sqrt(var(x) + eps)
//   g = dy w, xh = (x - mu) rstd
//   dx = rstd (g - mean(g) - xh mean(g xh)),  dw = sum_rows dy xh,
//   db = sum_rows dy
//
// Both passes are bound by DRAM: a row is read once into registers, its sums
// are formed there in fp32, and the result is written from the same registers.
// Forward, a warp takes a row (no barrier, and some twenty rows a SM in flight).
// The gradient also sums over rows: a CTA owns all columns of a row, each thread
// the same columns of every row that its CTA takes, so that the running dw and
// db stay in registers, and takes two rows between barriers.
//
// 65536 x 2560 bf16 forward: 114 us, 5.9 TB/s, 87% of a copy's rate.  Gradient of
// 32768 x 2560: 95 + 7 us, 5.1 TB/s (76%); its instructions take about as long as
// its loads.  33 x 2560: 5.7 us, two reductions' and three loads' latencies.
#include <algorithm>

#include "ops.h"
#include "rows.cuh"

namespace ittt {
namespace {

constexpr int kMaxWarps = 16;
constexpr int kMaxThreads = 32 * kMaxWarps;

// Statistics of a set of values: count, mean, sum of squared deviations.
// Merging two sets needs no second pass over the row and, unlike the sum of
// squares, loses nothing when the mean is large beside the spread.
struct Moments {
  float n, mean, m2;
};
__device__ __forceinline__ Moments merge(const Moments& a, const Moments& b) {
  const float n = a.n + b.n;
  const float f = n > 0.f ? b.n / n : 0.f;
  const float d = b.mean - a.mean;
  return Moments{n, a.mean + d * f, a.m2 + b.m2 + d * d * a.n * f};
}
__device__ __forceinline__ Moments shfl_xor(const Moments& a, int m) {
  return Moments{__shfl_xor_sync(~0u, a.n, m), __shfl_xor_sync(~0u, a.mean, m),
                 __shfl_xor_sync(~0u, a.m2, m)};
}

// The moments of the whole row in every thread; `buf` alternates between two
// rows' areas so that one barrier a row is enough.
__device__ __forceinline__ Moments block_moments(Moments a, Moments* buf) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
#pragma unroll
  for (int m = 16; m; m >>= 1) a = merge(a, shfl_xor(a, m));
  if (warps == 1) return a;
  if (lane == 0) buf[warp] = a;
  __syncthreads();
  Moments t = lane < warps ? buf[lane] : Moments{0.f, 0.f, 0.f};
#pragma unroll
  for (int m = 16; m; m >>= 1) t = merge(t, shfl_xor(t, m));
  return t;
}

__device__ __forceinline__ float2 block_sum2(float2 a, float2* buf) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
#pragma unroll
  for (int m = 16; m; m >>= 1) {
    a.x += __shfl_xor_sync(~0u, a.x, m);
    a.y += __shfl_xor_sync(~0u, a.y, m);
  }
  if (warps == 1) return a;
  if (lane == 0) buf[warp] = a;
  __syncthreads();
  float2 t = lane < warps ? buf[lane] : make_float2(0.f, 0.f);
#pragma unroll
  for (int m = 16; m; m >>= 1) {
    t.x += __shfl_xor_sync(~0u, t.x, m);
    t.y += __shfl_xor_sync(~0u, t.y, m);
  }
  return t;
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int m = 16; m; m >>= 1) x += __shfl_xor_sync(~0u, x, m);
  return x;
}

// Part of a row as read: 16 bytes (8 bf16 or 4 fp32 elements), or one element
// of a row that is not on a 16-byte boundary.
template <typename T, bool VEC>
struct Piece {
  static constexpr int N = 16 / sizeof(T);
  uint4 raw;
  __device__ __forceinline__ void clear() { raw = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void load(const T* p) { raw = __ldg(reinterpret_cast<const uint4*>(p)); }
  // unpacks anew: eight bf16 kept as fp32 between the passes over a row would
  // take twice the registers
  __device__ __forceinline__ void pin() {
    asm volatile("" : "+r"(raw.x), "+r"(raw.y), "+r"(raw.z), "+r"(raw.w));
  }
  __device__ __forceinline__ void get(float (&v)[N]) const {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 2) {
        const float2 f = unpack_bf16x2(w[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      } else {
        v[i] = __uint_as_float(w[i]);
      }
    }
  }
};
template <typename T>
struct Piece<T, false> {
  static constexpr int N = 1;
  float v0;
  __device__ __forceinline__ void clear() { v0 = 0.f; }
  __device__ __forceinline__ void pin() {}
  __device__ __forceinline__ void load(const T* p) {
    float v[1];
    RowVec<T, 1>::load(p, v);
    v0 = v[0];
  }
  __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = v0; }
};

// N elements of the weight or the bias from column c (a multiple of N).
template <typename W, int N>
__device__ __forceinline__ void load_param(const W* p, int64_t c, float (&v)[N]) {
  if constexpr (sizeof(W) == 2 && N == 4) {
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(p + c));
    const float2 lo = unpack_bf16x2(u.x), hi = unpack_bf16x2(u.y);
    v[0] = lo.x;
    v[1] = lo.y;
    v[2] = hi.x;
    v[3] = hi.y;
  } else {
    RowVec<W, N>::load(p + c, v);
  }
}

constexpr int kNormWarps = 4;

// A warp takes R neighbouring rows: lane l holds pieces l, l + 32, ... of each,
// as read.  The mean first, then the squared deviations from it: nothing cancels
// when the mean is large beside the spread.  W: type of weight and bias.
template <typename T, typename TO, typename W, bool VEC, int NV, int R>
__global__ void __launch_bounds__(32 * kNormWarps) layer_norm_kernel(NormArgs a, int nv) {
  using P = Piece<T, VEC>;
  constexpr int N = P::N;
  const T* x = static_cast<const T*>(a.x.data);
  const W* weight = static_cast<const W*>(a.weight);
  const W* bias = static_cast<const W*>(a.bias);
  TO* out = static_cast<TO*>(a.out);
  const int lane = threadIdx.x & 31;
  griddep_wait();
  griddep_launch_dependents();
  for (int64_t r0 = (int64_t(blockIdx.x) * kNormWarps + (threadIdx.x >> 5)) * R; r0 < a.N;
       r0 += int64_t(gridDim.x) * kNormWarps * R) {
    P p[R][NV];
    float mean[R], rstd[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const T* row = x + a.x.offset(r0 + i < a.N ? r0 + i : r0);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        p[i][j].clear();
        if (lane + 32 * j < nv) p[i][j].load(row + int64_t(lane + 32 * j) * N);
      }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      mean[i] = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float v[N], t = 0.f;
        p[i][j].get(v);
#pragma unroll
        for (int e = 0; e < N; ++e) t += v[e];
        mean[i] += t;
      }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) mean[i] = warp_sum(mean[i]) / float(a.d);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      rstd[i] = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (lane + 32 * j < nv) {
          float v[N], t = 0.f;
          p[i][j].pin();
          p[i][j].get(v);
#pragma unroll
          for (int e = 0; e < N; ++e) t += (v[e] - mean[i]) * (v[e] - mean[i]);
          rstd[i] += t;
        }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      rstd[i] = 1.f / sqrtf(warp_sum(rstd[i]) / float(a.d) + a.eps);
      if (lane == 0 && r0 + i < a.N) {
        if (a.mean) a.mean[r0 + i] = mean[i];
        if (a.rstd) a.rstd[r0 + i] = rstd[i];
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (lane + 32 * j < nv) {
        const int64_t c = int64_t(lane + 32 * j) * N;
        float w[N], b[N];
        load_param<W, N>(weight, c, w);
#pragma unroll
        for (int e = 0; e < N; ++e) b[e] = 0.f;
        if (bias) load_param<W, N>(bias, c, b);
#pragma unroll
        for (int i = 0; i < R; ++i)
          if (i == 0 || r0 + i < a.N) {
            float v[N];
            p[i][j].pin();
            p[i][j].get(v);
#pragma unroll
            for (int e = 0; e < N; ++e) v[e] = (v[e] - mean[i]) * rstd[i] * w[e] + b[e];
            RowVec<TO, N>::store(out + (r0 + i) * a.d + c, v);
          }
      }
  }
}

constexpr int kGradThreads = 384;

// Sums of V = 2, 4 or 8 numbers over the CTA, in every thread.  Within a warp by
// exchanging halves (each step leaves a lane half the numbers: 9 shuffles for
// eight numbers instead of 40); `buf` alternates between two areas so that one
// barrier a call is enough.
template <int V>
__device__ __forceinline__ void block_sums(float (&s)[V], float (*buf)[V]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  float x[V];
#pragma unroll
  for (int i = 0; i < V; ++i) x[i] = s[i];
  int m = 16;
#pragma unroll
  for (int cnt = V / 2; cnt >= 1; cnt >>= 1, m >>= 1) {
    const bool up = lane & m;
#pragma unroll
    for (int i = 0; i < cnt; ++i) {
      const float send = up ? x[i] : x[i + cnt], keep = up ? x[i + cnt] : x[i];
      x[i] = keep + __shfl_xor_sync(~0u, send, m);
    }
  }
  constexpr int G = 32 / V;  // neighbouring lanes that hold the same number
#pragma unroll
  for (int k = G / 2; k >= 1; k >>= 1) x[0] += __shfl_xor_sync(~0u, x[0], k);
  if (lane % G == 0) buf[warp][lane / G] = x[0];
  __syncthreads();
  float t = 0.f;
  for (int w = lane / V; w < warps; w += G) t += buf[w][lane % V];
#pragma unroll
  for (int k = V; k < 32; k <<= 1) t += __shfl_xor_sync(~0u, t, k);
#pragma unroll
  for (int i = 0; i < V; ++i) s[i] = __shfl_sync(~0u, t, i);
}

// (v - mean) rstd of two columns: the difference first, which is exact where the
// spread is small beside the mean.
__device__ __forceinline__ float2 centred(float2 v, float mean, float2 rstd) {
  return __fmul2_rn(__fadd2_rn(v, make_float2(-mean, -mean)), rstd);
}

// The rows that a CTA of the gradient reads ahead: stages of R rows of x and of
// dy in shared memory, filled by bulk copies that one thread issues.  With the
// loads in registers instead the rows in flight did not cover DRAM's latency
// (108 us at 32768 x 2560; 3 CTAs a SM at 56 registers).
constexpr int kMostStages = 4;
struct RowRing {
  uint64_t full[kMostStages];
  int abort;
};

// Thread t of the CTA owns pieces t, t + blockDim, ... (NV of them at most) of
// `nv`; groups of R neighbouring rows, blockIdx.x, + gridDim.x, ...  CTAS: at
// least so many a SM, so that one's loads run under another's reduction.  VEC:
// rows come through `stages` stages of shared memory.
template <typename T, bool VEC, int NV, int R, int THREADS, int CTAS>
__global__ void __launch_bounds__(THREADS, CTAS)
    layer_norm_grad_kernel(NormGradArgs a, int nv, bool wvec, int stages, unsigned int* status) {
  using P = Piece<T, VEC>;
  constexpr int N = P::N;
  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ RowRing bars;
  if (VEC && threadIdx.x == 0) {
    for (int i = 0; i < kMostStages; ++i) mbar_init(&bars.full[i], 1);
    bars.abort = 0;
    fence_mbar_init();
  }
  __shared__ float buf[2][THREADS / 32][2 * R];
  const T* x = static_cast<const T*>(a.x.data);
  const T* dy = static_cast<const T*>(a.dy.data);
  T* dx = static_cast<T*>(a.dx);
  griddep_wait();
  griddep_launch_dependents();
  constexpr int N2 = (N + 1) / 2;
  float2 w[NV][N2], dw[NV][N2], db[NV][N2];
  bool on[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int i = threadIdx.x + j * blockDim.x;
    on[j] = i < nv;
    float t[N];
#pragma unroll
    for (int e = 0; e < N; ++e) t[e] = 0.f;
    if (on[j]) {
      if (VEC && wvec && a.w_fp32)
        load_param<float, N>(static_cast<const float*>(a.weight), int64_t(i) * N, t);
      else
#pragma unroll
        for (int e = 0; e < N; ++e) t[e] = load_any(a.weight, a.w_fp32, int64_t(i) * N + e);
    }
#pragma unroll
    for (int e = 0; e < N2; ++e) {
      w[j][e] = make_float2(t[2 * e], 2 * e + 1 < N ? t[2 * e + 1 < N ? 2 * e + 1 : 0] : 0.f);
      dw[j][e] = db[j][e] = make_float2(0.f, 0.f);
    }
  }
  int par = 0, it = 0;
  const float inv = 1.f / float(a.d);
  const int64_t step = int64_t(gridDim.x) * R;
  const uint32_t row_bytes = uint32_t(a.d) * sizeof(T);
  auto fetch = [&](int stage, int64_t r0) {  // by one thread
    if (r0 >= a.N) return;
    const int rows = int(min(int64_t(R), a.N - r0));
    mbar_arrive_expect_tx(&bars.full[stage], 2 * rows * row_bytes);
    for (int i = 0; i < rows; ++i) {
      unsigned char* to = ring + size_t(stage * R + i) * 2 * row_bytes;
      bulk_load(to, x + a.x.offset(r0 + i), row_bytes, &bars.full[stage]);
      bulk_load(to + row_bytes, dy + a.dy.offset(r0 + i), row_bytes, &bars.full[stage]);
    }
  };
  if constexpr (VEC) {
    __syncthreads();
    if (threadIdx.x == 0)
      for (int i = 0; i < stages; ++i) fetch(i, int64_t(blockIdx.x) * R + i * step);
  }
  for (int64_t r0 = int64_t(blockIdx.x) * R; r0 < a.N; r0 += step, par ^= 1, ++it) {
    const int stage = it % stages;
    bool loaded = true;
    if (VEC && !(loaded = mbar_wait(&bars.full[stage], (it / stages) & 1, &bars.abort)))
      raise_abort(&bars.abort, status, kStatusTimeout);
    P px[R][NV], pg[R][NV];
    float mean[R], rstd[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int64_t r = r0 + i;
      mean[i] = rstd[i] = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        px[i][j].clear();
        pg[i][j].clear();
      }
      if (r < a.N) {
        const T* xr = x + a.x.offset(r);
        const T* gr = dy + a.dy.offset(r);
        mean[i] = __ldg(a.mean + r);
        rstd[i] = __ldg(a.rstd + r);
#pragma unroll
        for (int j = 0; j < NV; ++j)
          if (on[j]) {
            const int64_t c = int64_t(threadIdx.x + j * blockDim.x) * N;
            if constexpr (VEC) {
              const unsigned char* row = ring + size_t(stage * R + i) * 2 * row_bytes + c * sizeof(T);
              px[i][j].raw = *reinterpret_cast<const uint4*>(row);
              pg[i][j].raw = *reinterpret_cast<const uint4*>(row + row_bytes);
            } else {
              px[i][j].load(xr + c);
              pg[i][j].load(gr + c);
            }
          }
      }
    }
    float s[2 * R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      // two columns an instruction where a piece has them
      float2 sg = make_float2(0.f, 0.f), sx = sg;
      const float2 mul = make_float2(rstd[i], rstd[i]);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float v[N], g[N];
        px[i][j].get(v);
        pg[i][j].get(g);
#pragma unroll
        for (int e = 0; e < N; e += 2) {
          const bool one = N == 1;
          const float2 v2 = make_float2(v[e], one ? 0.f : v[one ? 0 : e + 1]);
          const float2 g2 = make_float2(g[e], one ? 0.f : g[one ? 0 : e + 1]);
          const float2 xh = centred(v2, mean[i], mul), gw = __fmul2_rn(g2, w[j][e / 2]);
          dw[j][e / 2] = __ffma2_rn(g2, xh, dw[j][e / 2]);
          db[j][e / 2] = __fadd2_rn(g2, db[j][e / 2]);
          sg = __fadd2_rn(gw, sg);
          sx = __ffma2_rn(gw, xh, sx);
        }
      }
      s[2 * i] = sg.x + sg.y;
      s[2 * i + 1] = sx.x + sx.y;
    }
    block_sums<2 * R>(s, buf[par]);
    // every thread is past the barrier: the stage is read
    if (VEC && threadIdx.x == 0 && loaded) fetch(stage, r0 + stages * step);
    if (dx == nullptr) continue;
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (r0 + i < a.N) {
        const float c1 = -rstd[i] * s[2 * i] * inv, c2 = -rstd[i] * s[2 * i + 1] * inv;
        const float2 mul = make_float2(rstd[i], rstd[i]);
#pragma unroll
        for (int j = 0; j < NV; ++j)
          if (on[j]) {
            float v[N], g[N];
            px[i][j].pin();
            pg[i][j].pin();
            px[i][j].get(v);
            pg[i][j].get(g);
#pragma unroll
            for (int e = 0; e < N; e += 2) {
              const bool one = N == 1;
              const float2 v2 = make_float2(v[e], one ? 0.f : v[one ? 0 : e + 1]);
              const float2 g2 = make_float2(g[e], one ? 0.f : g[one ? 0 : e + 1]);
              // rstd g w - rstd mean(g w) - rstd mean(g w xh) xh
              const float2 t = __ffma2_rn(make_float2(c2, c2), centred(v2, mean[i], mul), make_float2(c1, c1));
              const float2 o = __ffma2_rn(__fmul2_rn(g2, w[j][e / 2]), mul, t);
              v[e] = o.x;
              if (!one) v[one ? 0 : e + 1] = o.y;
            }
            RowVec<T, N>::store(dx + (r0 + i) * a.d + int64_t(threadIdx.x + j * blockDim.x) * N, v);
          }
      }
  }
  if (VEC) settle(&bars.abort);
  // This CTA's share of dw and db: [2][gridDim.x][d].
  if (a.dw == nullptr && a.db == nullptr) return;
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (on[j]) {
      const int64_t c = int64_t(threadIdx.x + j * blockDim.x) * N;
      float t[N];
#pragma unroll
      for (int e = 0; e < N; ++e) t[e] = e & 1 ? dw[j][e / 2].y : dw[j][e / 2].x;
      RowVec<float, N>::store(a.ws + int64_t(blockIdx.x) * a.d + c, t);
#pragma unroll
      for (int e = 0; e < N; ++e) t[e] = e & 1 ? db[j][e / 2].y : db[j][e / 2].x;
      RowVec<float, N>::store(a.ws + (int64_t(gridDim.x) + blockIdx.x) * a.d + c, t);
    }
}

// Adds the CTAs' shares in their order: 32 columns by 32 groups of shares a
// CTA, the groups joined in a fixed order (no atomics: the same sum in every
// call).  blockIdx.y: 0 dw, 1 db.
__global__ void __launch_bounds__(1024) column_sum_kernel(const float* part, int parts, int64_t d,
                                                          void* dw, bool dw_fp32, void* db,
                                                          bool db_fp32) {
  __shared__ float acc[32][33];
  griddep_wait();
  griddep_launch_dependents();
  void* out = blockIdx.y ? db : dw;
  if (out == nullptr) return;
  const float* src = part + int64_t(blockIdx.y) * parts * d;
  const int64_t c = int64_t(blockIdx.x) * 32 + threadIdx.x;
  float s = 0.f;
  if (c < d)
#pragma unroll 4
    for (int p = threadIdx.y; p < parts; p += 32) s += src[int64_t(p) * d + c];
  acc[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  s = acc[threadIdx.x][threadIdx.y];  // column threadIdx.y, group threadIdx.x
#pragma unroll
  for (int m = 16; m; m >>= 1) s += __shfl_xor_sync(~0u, s, m);
  const int64_t col = int64_t(blockIdx.x) * 32 + threadIdx.y;
  if (threadIdx.x == 0 && col < d) store_any(out, blockIdx.y ? db_fp32 : dw_fp32, col, s);
}

// Few rows, rows that are not on 16-byte boundaries, or too wide for a warp: a CTA
// a row, its elements in registers, K a thread.  Element by element the load and
// store instructions bound it: 16384 x 2305 bf16 in 78 us (1.9 TB/s), fp32 in 74
// (4.1 TB/s); by warps of 96 elements a lane 143 and 162 us, by three passes over
// the row 205 and 252.
constexpr int kRowThreads = 256;
template <typename T, typename TO, typename W, int K>
__global__ void __launch_bounds__(kRowThreads) layer_norm_row_kernel(NormArgs a) {
  __shared__ float2 buf[4][kMaxWarps];
  const W* weight = static_cast<const W*>(a.weight);
  const W* bias = static_cast<const W*>(a.bias);
  const T* x = static_cast<const T*>(a.x.data);
  TO* out = static_cast<TO*>(a.out);
  griddep_wait();
  griddep_launch_dependents();
  int par = 0;
  for (int64_t r = blockIdx.x; r < a.N; r += gridDim.x, par ^= 2) {
    const T* row = x + a.x.offset(r);
    float v[K];
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < K; ++j) {
      const int c = threadIdx.x + j * kRowThreads;
      v[j] = 0.f;
      if (c < a.d) {
        float t[1];
        RowVec<T, 1>::load(row + c, t);
        v[j] = t[0];
      }
    }
#pragma unroll
    for (int j = 0; j < K; ++j) s.x += v[j];
    const float mean = block_sum2(s, buf[par]).x / float(a.d);
    s.x = 0.f;
#pragma unroll
    for (int j = 0; j < K; ++j) {
      v[j] -= mean;
      s.x += int(threadIdx.x) + j * kRowThreads < a.d ? v[j] * v[j] : 0.f;
    }
    const float rstd = 1.f / sqrtf(block_sum2(s, buf[par + 1]).x / float(a.d) + a.eps);
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[r] = mean;
      if (a.rstd) a.rstd[r] = rstd;
    }
    // four at a time: their loads of the weight and the bias go out together
#pragma unroll
    for (int j0 = 0; j0 < K; j0 += 4) {
      float w[4], b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = threadIdx.x + (j0 + j) * kRowThreads;
        w[j] = b[j] = 0.f;
        if (c < a.d) load_param<W, 1>(weight, c, reinterpret_cast<float(&)[1]>(w[j]));
        if (c < a.d && bias) load_param<W, 1>(bias, c, reinterpret_cast<float(&)[1]>(b[j]));
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = threadIdx.x + (j0 + j) * kRowThreads;
        const float y[1] = {v[j0 + j] * rstd * w[j] + b[j]};
        if (c < a.d) RowVec<TO, 1>::store(out + r * a.d + c, y);
      }
    }
  }
}

// Rows too wide for the registers: element by
// element, the row read again, through L1 and L2, for each pass over it.
template <typename T, typename TO>
__global__ void __launch_bounds__(kMaxThreads) layer_norm_wide_kernel(NormArgs a) {
  __shared__ Moments buf[2][kMaxWarps];
  const T* x = static_cast<const T*>(a.x.data);
  TO* out = static_cast<TO*>(a.out);
  griddep_wait();
  griddep_launch_dependents();
  int par = 0;
  for (int64_t r = blockIdx.x; r < a.N; r += gridDim.x, par ^= 1) {
    const T* row = x + a.x.offset(r);
    Moments m{0.f, 0.f, 0.f};
    for (int64_t c = threadIdx.x; c < a.d; c += blockDim.x) {
      float v[1];
      RowVec<T, 1>::load(row + c, v);
      m.n += 1.f;
      const float dlt = v[0] - m.mean;
      m.mean += dlt / m.n;
      m.m2 += dlt * (v[0] - m.mean);
    }
    m = block_moments(m, buf[par]);
    const float rstd = 1.f / sqrtf(m.m2 / float(a.d) + a.eps);
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[r] = m.mean;
      if (a.rstd) a.rstd[r] = rstd;
    }
    for (int64_t c = threadIdx.x; c < a.d; c += blockDim.x) {
      float v[1];
      RowVec<T, 1>::load(row + c, v);
      v[0] = (v[0] - m.mean) * rstd * load_any(a.weight, a.w_fp32, c) +
             (a.bias ? load_any(a.bias, a.b_fp32, c) : 0.f);
      RowVec<TO, 1>::store(out + r * a.d + c, v);
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kMaxThreads) layer_norm_grad_wide_kernel(NormGradArgs a) {
  __shared__ float2 buf[2][kMaxWarps];
  const T* x = static_cast<const T*>(a.x.data);
  const T* dy = static_cast<const T*>(a.dy.data);
  T* dx = static_cast<T*>(a.dx);
  griddep_wait();
  griddep_launch_dependents();
  const bool sums = a.dw != nullptr || a.db != nullptr;
  float* dw = a.ws + int64_t(blockIdx.x) * a.d;  // this CTA's shares, in place
  float* db = a.ws + (int64_t(gridDim.x) + blockIdx.x) * a.d;
  bool first = true;
  int par = 0;
  for (int64_t r = blockIdx.x; r < a.N; r += gridDim.x, par ^= 1, first = false) {
    const T* xr = x + a.x.offset(r);
    const T* gr = dy + a.dy.offset(r);
    const float mu = a.mean[r], rstd = a.rstd[r];
    float2 s = make_float2(0.f, 0.f);
    for (int64_t c = threadIdx.x; c < a.d; c += blockDim.x) {
      float v[1], g[1];
      RowVec<T, 1>::load(xr + c, v);
      RowVec<T, 1>::load(gr + c, g);
      const float xh = (v[0] - mu) * rstd, gw = g[0] * load_any(a.weight, a.w_fp32, c);
      s.x += gw;
      s.y += gw * xh;
      if (sums) {
        dw[c] = (first ? 0.f : dw[c]) + g[0] * xh;
        db[c] = (first ? 0.f : db[c]) + g[0];
      }
    }
    s = block_sum2(s, buf[par]);
    const float c1 = s.x / float(a.d), c2 = s.y / float(a.d);
    if (dx != nullptr)
      for (int64_t c = threadIdx.x; c < a.d; c += blockDim.x) {
        float v[1], g[1];
        RowVec<T, 1>::load(xr + c, v);
        RowVec<T, 1>::load(gr + c, g);
        v[0] = rstd * (g[0] * load_any(a.weight, a.w_fp32, c) - c1 - (v[0] - mu) * rstd * c2);
        RowVec<T, 1>::store(dx + r * a.d + c, v);
      }
  }
}

// Shares of dw and db: at most this many CTAs walk the rows.
constexpr int64_t kMaxShares = 1024;

// CTAs that walk N groups of rows: as many as are resident at once.
template <typename... KArgs>
int64_t row_grid(void (*kernel)(KArgs...), int threads, int64_t N, int num_sms, cudaError_t* e) {
  if (N <= num_sms) {  // one each: nothing to look up
    *e = cudaSuccess;
    return N;
  }
  int resident = 0;
  *e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&resident, kernel, threads, 0);
  return std::min(std::min<int64_t>(N, kMaxShares), int64_t(std::max(resident, 1)) * num_sms);
}

template <typename T, typename TO, typename W, bool VEC, int NV, int R>
cudaError_t run_norm(const LaunchEnv& env, const NormArgs& a) {
  const int64_t groups = (a.N + R * kNormWarps - 1) / (R * kNormWarps);
  return launch_pdl(layer_norm_kernel<T, TO, W, VEC, NV, R>,
                    dim3(unsigned(std::min<int64_t>(groups, int64_t(env.num_sms) * 64))),
                    dim3(32 * kNormWarps), 0, env.stream, a, int(a.d / Piece<T, VEC>::N));
}

template <typename T, typename TO, typename W, int K>
cudaError_t run_norm_row(const LaunchEnv& env, const NormArgs& a) {
  cudaError_t e;
  const int64_t grid = row_grid(layer_norm_row_kernel<T, TO, W, K>, kRowThreads, a.N, env.num_sms, &e);
  if (e != cudaSuccess) return e;
  return launch_pdl(layer_norm_row_kernel<T, TO, W, K>, dim3(unsigned(grid)), dim3(kRowThreads), 0, env.stream, a);
}

template <typename T, typename TO, typename W>
cudaError_t pick_norm(const LaunchEnv& env, const NormArgs& a) {
  constexpr int N = 16 / sizeof(T);
  if (!a.bias || a.b_fp32 == a.w_fp32) {
    // A warp a row keeps DRAM busy once rows are many; with few of them a CTA a row
    // has the shorter path.  us by warp / by CTA, bf16: 40 x 2560 12 / 8,
    // 600 x 5120 18 / 14, 1000 x 5120 18 / 20, 2000 x 2560 12 / 16,
    // 40 x 1024 8 / 8, 40 x 512 6 / 6, 16384 x 2560 39 / 90.
    const bool few = a.N <= 5 * env.num_sms && a.d * int64_t(sizeof(T)) >= 4096;
    // d % 8 == 0 keeps every dense row, of either type, on a 16-byte boundary
    if (!few && a.d % 8 == 0 && rows_aligned(a.x.data, a.x.stride_b, a.x.stride_t, a.x.fp32) &&
        aligned16(a.out) && aligned16(a.weight) && (!a.bias || aligned16(a.bias))) {
      const int64_t nv = a.d / N;
      // pieces a lane, unrolled: with the next step up instead, 16384 x 2568 bf16
      // takes 63 us (not 49), 4096 80 (74), 4096 fp32 by CTAs 367 (102)
      if (nv <= 32 * 2) return run_norm<T, TO, W, true, 2, 1>(env, a);
      if (nv <= 32 * 5) return run_norm<T, TO, W, true, 5, 1>(env, a);
      if (nv <= 32 * 10) return run_norm<T, TO, W, true, 10, 1>(env, a);
      if (nv <= 32 * 16) return run_norm<T, TO, W, true, 16, 1>(env, a);
      if (nv <= 32 * 20) return run_norm<T, TO, W, true, 20, 1>(env, a);
      if (nv <= 32 * 32) return run_norm<T, TO, W, true, 32, 1>(env, a);
      if (nv <= 32 * 40) return run_norm<T, TO, W, true, 40, 1>(env, a);
    } else if (a.d <= 32 * 12) {
      return run_norm<T, TO, W, false, 12, 1>(env, a);
    }
    if (a.d <= 8 * kRowThreads) return run_norm_row<T, TO, W, 8>(env, a);
    if (a.d <= 12 * kRowThreads) return run_norm_row<T, TO, W, 12>(env, a);
    if (a.d <= 20 * kRowThreads) return run_norm_row<T, TO, W, 20>(env, a);
    if (a.d <= 40 * kRowThreads) return run_norm_row<T, TO, W, 40>(env, a);
  }
  cudaError_t e;
  const int64_t grid =
      row_grid(layer_norm_wide_kernel<T, TO>, kMaxThreads, a.N, env.num_sms, &e);
  if (e != cudaSuccess) return e;
  return launch_pdl(layer_norm_wide_kernel<T, TO>, dim3(unsigned(grid)), dim3(kMaxThreads), 0,
                    env.stream, a);
}

template <typename T, bool VEC, int NV, int R, int THREADS, int CTAS>
cudaError_t run_norm_grad(const LaunchEnv& env, const NormGradArgs& a, int64_t* grid, bool wvec) {
  const auto kernel = layer_norm_grad_kernel<T, VEC, NV, R, THREADS, CTAS>;
  const int nv = int(a.d / Piece<T, VEC>::N);
  const int threads = ((nv + NV - 1) / NV + 31) / 32 * 32;
  const size_t stage = VEC ? size_t(R) * 2 * size_t(a.d) * sizeof(T) : 0;
  // what CTAS CTAs a SM leave each (a stage of the widest row fits)
  const size_t room = size_t(216) * 1024 / CTAS;
  const int stages = VEC ? int(std::min<size_t>(kMostStages, room / stage)) : 1;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(room));
  if (e != cudaSuccess) return e;
  const int64_t groups = (a.N + R - 1) / R;
  int resident = 1;
  if (groups > env.num_sms) {
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&resident, kernel, threads, stages * stage);
    if (e != cudaSuccess) return e;
  }
  *grid = std::min(std::min(groups, kMaxShares), int64_t(std::max(resident, 1)) * env.num_sms);
  return launch_pdl(kernel, dim3(unsigned(*grid)), dim3(threads), stages * stage, env.stream, a, nv, wvec,
                    stages, env.status);
}

template <typename T>
cudaError_t pick_norm_grad(const LaunchEnv& env, const NormGradArgs& a, int64_t* grid) {
  if (a.d % 8 == 0 && rows_aligned(a.x.data, a.x.stride_b, a.x.stride_t, a.x.fp32) &&
      rows_aligned(a.dy.data, a.dy.stride_b, a.dy.stride_t, a.dy.fp32) && aligned16(a.dx)) {
    const int64_t nv = a.d / (16 / sizeof(T));
    const bool wvec = aligned16(a.weight);
    if (nv <= 2 * 192) return run_norm_grad<T, true, 2, 2, 192, 3>(env, a, grid, wvec);
    if (nv <= 2 * kGradThreads) return run_norm_grad<T, true, 2, 2, kGradThreads, 1>(env, a, grid, wvec);
    if (nv <= 4 * kGradThreads) return run_norm_grad<T, true, 4, 1, kGradThreads, 1>(env, a, grid, wvec);
    if (nv <= 6 * kGradThreads) return run_norm_grad<T, true, 6, 1, kGradThreads, 1>(env, a, grid, wvec);
  } else {
    if (a.d <= 4 * kGradThreads) return run_norm_grad<T, false, 4, 2, kGradThreads, 2>(env, a, grid, false);
    // beyond that the rows in flight count: at 16384 x 1537 / 2305 / 4607 bf16 two
    // CTAs of 384 threads with a row each take 106 / 152 / 404 us, one of 768 with
    // two rows 139 / 156 / 309
    if (a.d <= 6 * kGradThreads) return run_norm_grad<T, false, 6, 1, kGradThreads, 2>(env, a, grid, false);
    if (a.d <= 4 * 768) return run_norm_grad<T, false, 4, 2, 768, 1>(env, a, grid, false);
    if (a.d <= 7 * 768) return run_norm_grad<T, false, 7, 2, 768, 1>(env, a, grid, false);
  }
  cudaError_t e;
  *grid = row_grid(layer_norm_grad_wide_kernel<T>, kMaxThreads, a.N, env.num_sms, &e);
  if (e != cudaSuccess) return e;
  return launch_pdl(layer_norm_grad_wide_kernel<T>, dim3(unsigned(*grid)), dim3(kMaxThreads), 0,
                    env.stream, a);
}

}  // namespace

cudaError_t launch_layer_norm(const LaunchEnv& env, const NormArgs& a) {
  using H = __nv_bfloat16;
  if (a.w_fp32) {
    if (a.x.fp32) return a.out_fp32 ? pick_norm<float, float, float>(env, a) : pick_norm<float, H, float>(env, a);
    return a.out_fp32 ? pick_norm<H, float, float>(env, a) : pick_norm<H, H, float>(env, a);
  }
  if (a.x.fp32) return a.out_fp32 ? pick_norm<float, float, H>(env, a) : pick_norm<float, H, H>(env, a);
  return a.out_fp32 ? pick_norm<H, float, H>(env, a) : pick_norm<H, H, H>(env, a);
}

size_t layer_norm_grad_scratch(int64_t N, int64_t d) {
  return size_t(std::min<int64_t>(N, kMaxShares)) * size_t(d) * 2 * sizeof(float);
}

cudaError_t launch_layer_norm_grad(const LaunchEnv& env, const NormGradArgs& a) {
  int64_t grid = 0;
  cudaError_t e = a.x.fp32 ? pick_norm_grad<float>(env, a, &grid)
                           : pick_norm_grad<__nv_bfloat16>(env, a, &grid);
  if (e != cudaSuccess || (a.dw == nullptr && a.db == nullptr)) return e;
  return launch_pdl(column_sum_kernel, dim3(unsigned((a.d + 31) / 32), 2), dim3(32, 32), 0,
                    env.stream, static_cast<const float*>(a.ws), int(grid), a.d, a.dw, a.dw_fp32,
                    a.db, a.db_fp32);
}

}  // namespace ittt
