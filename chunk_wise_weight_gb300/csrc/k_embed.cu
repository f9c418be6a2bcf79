// k_embed.cu -- embedding lookup with scaling, and its gradient.
//
//   Y[n] = scale E[id[n]]          dE[r] = scale sum_{n: id[n] = r} dY[n]
//
// An id outside [0, V) is padding: its row of Y is zero and its row of dY is
// dropped.  Both directions only move rows, so DRAM bounds them.
//
// The gradient sums each row's terms in fp32, without atomics on floats, in an
// order that the ids alone fix: the same bits in every call.  The ids are
// sorted, stably, with their positions (by one cluster of CTAs, beside the
// CTAs that zero the table); tiles of sorted positions are then summed, each
// distinct id a run of neighbours.  A run inside one tile is written at once;
// a run that crosses tiles leaves a partial sum in each of them, and the tile
// where it begins joins them: in order, or for a long run as eight sums of every
// eighth part, added in order.  So a token that fills half the batch costs no more
// than tokens that occur once.
//
// Lookup of 65536 rows of 2560 bf16: 66 us, 6.6 TB/s, a copy's rate.  Gradient of
// 16381 rows into a zeroed 65536 x 2560 fp32 table: 116 (the fill, the sort beside
// it) + 29 + 14 us, 72% of a copy's rate.  32768 rows of 2048 added to an fp32
// table: 24 (sort) + 62 + 23 us; the rows' latencies and the joins of frequent
// tokens' runs bound it.
#include <algorithm>

#include <cooperative_groups.h>

#include "ops.h"
#include "rows.cuh"

namespace ittt {
namespace {

namespace cg = cooperative_groups;

// ------------------------------------------------------------------- lookup
constexpr int kLookupWarps = 8;
constexpr int kLookupVecs = 4;  // vectors a lane, all in flight together

// A warp copies 32 * kLookupVecs vectors of one row: enough loads in flight
// to cover the latency of a random row, and several warps a row when rows are
// few.
template <typename T, typename TO, int VEC>
__global__ void __launch_bounds__(32 * kLookupWarps) embed_kernel(EmbedArgs a, int nv) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t n = int64_t(blockIdx.x) * kLookupWarps + (threadIdx.x >> 5);
  if (n >= a.N) return;
  const int64_t id = load_id(a.ids, a.ids64, n);
  const bool in = id >= 0 && id < a.V;
  const T* src = static_cast<const T*>(a.table) + (in ? id : 0) * a.d;
  TO* dst = static_cast<TO*>(a.out) + n * a.d;
  const int v0 = blockIdx.y * 32 * kLookupVecs + (threadIdx.x & 31);
  float v[kLookupVecs][VEC];
#pragma unroll
  for (int j = 0; j < kLookupVecs; ++j) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[j][e] = 0.f;
    if (in && v0 + 32 * j < nv) RowVec<T, VEC>::load(src + int64_t(v0 + 32 * j) * VEC, v[j]);
  }
#pragma unroll
  for (int j = 0; j < kLookupVecs; ++j)
    if (v0 + 32 * j < nv) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[j][e] = in ? v[j][e] * a.scale : 0.f;
      RowVec<TO, VEC>::store(dst + int64_t(v0 + 32 * j) * VEC, v[j]);
    }
}

template <typename T, typename TO>
cudaError_t run_embed(const LaunchEnv& env, const EmbedArgs& a) {
  constexpr int V = sizeof(T) == 2 ? 8 : 4;
  const unsigned gx = unsigned((a.N + kLookupWarps - 1) / kLookupWarps);
  auto grid = [&](int64_t nv) {
    return dim3(gx, unsigned((nv + 32 * kLookupVecs - 1) / (32 * kLookupVecs)));
  };
  // d % 8 == 0 keeps every row of either type on a 16-byte boundary
  if (a.d % 8 == 0 && aligned16(a.table) && aligned16(a.out))
    return launch_pdl(embed_kernel<T, TO, V>, grid(a.d / V), dim3(32 * kLookupWarps), 0,
                      env.stream, a, int(a.d / V));
  return launch_pdl(embed_kernel<T, TO, 1>, grid(a.d), dim3(32 * kLookupWarps), 0, env.stream, a,
                    int(a.d));
}

// --------------------------------------------------------- sort of the ids
constexpr int kSortCtas = 8;        // one cluster
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxBits = 9;         // bits of one pass
constexpr int kBins = 1 << kMaxBits;
constexpr int kSortAhead = 8;       // elements a lane loads together

struct SortArgs {
  const void* ids;
  bool ids64;
  int64_t N, V;
  int bits, passes;  // bits a pass
  int* key[2];       // the result is in key[(passes - 1) & 1], pos[...]
  int* pos[2];
  uint4* fill;       // table to zero, or nullptr
  int64_t fill_vecs;
  int fill_tail;     // bytes after the last whole vector
};

// Clusters after the first zero the table.  The first sorts (id, position)
// by least-significant digits: every warp owns a contiguous span of the
// input, counts its digits, learns from the other warps and CTAs (distributed
// shared memory) where its elements of each digit go, and walks the span
// again, 32 at a time in order, so equal digits keep their order.
__global__ void __cluster_dims__(kSortCtas, 1, 1) __launch_bounds__(kSortThreads)
    sort_ids_kernel(SortArgs a) {
  extern __shared__ int smem[];
  int* count = smem;                                 // [kSortWarps][kBins]
  int* total = smem + kSortWarps * kBins;            // [kBins] this CTA's count a digit
  int* warp_sum = total + kBins;                     // [kSortWarps]
  griddep_wait();
  griddep_launch_dependents();
  if (blockIdx.x >= kSortCtas) {
    const int64_t step = int64_t(gridDim.x - kSortCtas) * kSortThreads;
    int64_t i = int64_t(blockIdx.x - kSortCtas) * kSortThreads + threadIdx.x;
    const uint4 z = make_uint4(0, 0, 0, 0);
    for (; i < a.fill_vecs; i += step) a.fill[i] = z;
    if (blockIdx.x == kSortCtas && threadIdx.x < unsigned(a.fill_tail))
      reinterpret_cast<unsigned char*>(a.fill + a.fill_vecs)[threadIdx.x] = 0;
    return;
  }
  cg::cluster_group cluster = cg::this_cluster();
  const int cta = int(cluster.block_rank()), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t span = ((a.N + kSortCtas * kSortWarps - 1) / (kSortCtas * kSortWarps) + 31) / 32 * 32;
  const int64_t lo = min(a.N, span * (int64_t(cta) * kSortWarps + warp));
  const int64_t hi = min(a.N, lo + span);
  const int bins = 1 << a.bits;
  int* mine = count + warp * kBins;
  for (int pass = 0; pass < a.passes; ++pass) {
    const int shift = pass * a.bits;
    const int* key_in = a.key[(pass + 1) & 1];
    const int* pos_in = a.pos[(pass + 1) & 1];
    auto load = [&](int64_t i) {
      if (pass == 0) {
        const int64_t id = load_id(a.ids, a.ids64, i);
        return id >= 0 && id < a.V ? int(id) : int(a.V);  // padding sorts last
      }
      return __ldcg(key_in + i);  // written by the other CTAs of the cluster
    };
    for (int b = lane; b < bins; b += 32) mine[b] = 0;
    __syncwarp();
    for (int64_t i0 = lo + lane; i0 < hi; i0 += 32 * kSortAhead) {
      int key[kSortAhead];
#pragma unroll
      for (int j = 0; j < kSortAhead; ++j) key[j] = i0 + 32 * j < hi ? load(i0 + 32 * j) : -1;
#pragma unroll
      for (int j = 0; j < kSortAhead; ++j)
        if (key[j] >= 0) atomicAdd(mine + ((key[j] >> shift) & (bins - 1)), 1);
    }
    __syncthreads();
    // per digit: each warp's elements before it in this CTA, and the CTA's total
    for (int b = threadIdx.x; b < bins; b += kSortThreads) {
      int c[kSortWarps], s = 0;
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) c[w] = count[w * kBins + b];
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) {
        count[w * kBins + b] = s;
        s += c[w];
      }
      total[b] = s;
    }
    cluster.sync();
    // first slot of each digit (bins <= 512 <= threads), then this CTA's share of it
    int all = 0, before = 0;
    if (threadIdx.x < unsigned(bins))
      for (int c = 0; c < kSortCtas; ++c) {
        const int v = cluster.map_shared_rank(total, c)[threadIdx.x];
        before += c < cta ? v : 0;
        all += v;
      }
    int scan = all;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const int v = __shfl_up_sync(~0u, scan, m);
      if (lane >= m) scan += v;
    }
    if (lane == 31) warp_sum[warp] = scan;
    __syncthreads();
    if (threadIdx.x < unsigned(bins)) {
      int base = scan - all + before;
      for (int w = 0; w < warp; ++w) base += warp_sum[w];
      int c[kSortWarps];
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) c[w] = count[w * kBins + threadIdx.x];
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) count[w * kBins + threadIdx.x] = c[w] + base;
    }
    __syncthreads();
    int* key_out = a.key[pass & 1];
    int* pos_out = a.pos[pass & 1];
    for (int64_t i0 = lo + lane; i0 - lane < hi; i0 += 32 * kSortAhead) {
      int keys[kSortAhead], at_pos[kSortAhead];
#pragma unroll
      for (int j = 0; j < kSortAhead; ++j) {
        const int64_t i = i0 + 32 * j;
        keys[j] = i < hi ? load(i) : -1;
        at_pos[j] = i < hi ? (pass == 0 ? int(i) : __ldcg(pos_in + i)) : 0;
      }
#pragma unroll
      for (int j = 0; j < kSortAhead; ++j) {
        const bool in = keys[j] >= 0;
        if (!__any_sync(~0u, in)) break;
        const int digit = in ? (keys[j] >> shift) & (bins - 1) : -1;
        const unsigned peers = __match_any_sync(~0u, digit);
        int at = in ? mine[digit] : 0;
        __syncwarp();
        at += __popc(peers & ((1u << lane) - 1));
        if (in) {
          key_out[at] = keys[j];
          pos_out[at] = at_pos[j];
          if ((peers >> lane) == 1u) mine[digit] = at + 1;  // the last of its peers
        }
        __syncwarp();
      }
    }
    __threadfence();
    cluster.sync();  // also keeps `total` until every CTA has read it
  }
}

// ------------------------------------------------------ sums of sorted rows
// Sorted positions a tile.  All rows of a tile are loaded at once (and, when
// adding, the rows of the table that it finishes), so a tile costs one latency;
// a longer tile would keep more registers, a shorter one leave more partial
// sums.
constexpr int kTile = 16;
constexpr int kSumThreads = 128;

struct SumArgs {
  const int* key;  // sorted ids, padding (V) last
  const int* pos;
  int64_t N, V, d;
  RowView dy;
  float scale;
  void* grad;
  bool grad_fp32;
  float* part;  // [tiles][2][d]: run from the tile before, run into the next
};

// VEC (4 or 1) elements of a row as read.
template <typename T, int VEC>
struct Terms;
template <>
struct Terms<__nv_bfloat16, 4> {
  uint2 raw;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { raw = __ldg(reinterpret_cast<const uint2*>(p)); }
  __device__ __forceinline__ void add_to(float (&acc)[4]) const {
    const float2 lo = unpack_bf16x2(raw.x), hi = unpack_bf16x2(raw.y);
    acc[0] += lo.x;
    acc[1] += lo.y;
    acc[2] += hi.x;
    acc[3] += hi.y;
  }
};
template <>
struct Terms<float, 4> {
  float4 raw;
  __device__ __forceinline__ void load(const float* p) { raw = __ldg(reinterpret_cast<const float4*>(p)); }
  __device__ __forceinline__ void add_to(float (&acc)[4]) const {
    acc[0] += raw.x;
    acc[1] += raw.y;
    acc[2] += raw.z;
    acc[3] += raw.w;
  }
};
template <typename T>
struct Terms<T, 1> {
  T raw;
  __device__ __forceinline__ void load(const T* p) { raw = *p; }
  __device__ __forceinline__ void add_to(float (&acc)[1]) const { acc[0] += float(raw); }
};

// blockIdx.x: tile; blockIdx.y: kSumThreads * VEC columns.  ADD: into an fp32
// table; the old values are read with plain loads, since no other tile of this
// launch writes a row that this one finishes.
template <typename T, int VEC, bool ADD>
__global__ void __launch_bounds__(kSumThreads) sum_rows_kernel(SumArgs a, int nv) {
  __shared__ int key[kTile + 2];  // with the neighbours on both sides
  __shared__ int64_t off[kTile];
  griddep_wait();
  griddep_launch_dependents();
  const int64_t p0 = int64_t(blockIdx.x) * kTile;
  const int n = int(min(int64_t(kTile), a.N - p0));
  if (threadIdx.x < kTile + 2) {
    const int i = threadIdx.x;
    const int64_t p = p0 + i - 1;
    key[i] = p >= 0 && i <= n + 1 && p < a.N ? a.key[p] : -1;
    if (i >= 1 && i <= n) off[i - 1] = a.dy.offset(a.pos[p]);
  }
  __syncthreads();
  const int vi = blockIdx.y * kSumThreads + threadIdx.x;
  if (vi >= nv) return;
  const int64_t c = int64_t(vi) * VEC;
  const T* dy = static_cast<const T*>(a.dy.data) + c;
  Terms<T, VEC> v[kTile];
  float old[ADD ? kTile : 1][VEC];
#pragma unroll
  for (int i = 0; i < kTile; ++i)
    if (i < n && key[i + 1] < a.V) v[i].load(dy + off[i]);
  if constexpr (ADD) {
#pragma unroll
    for (int i = 0; i < kTile; ++i)
      if (i < n && key[i + 1] < a.V && key[i + 2] != key[i + 1]) {
        const float* g = static_cast<const float*>(a.grad) + int64_t(key[i + 1]) * a.d + c;
        if constexpr (VEC == 4)
          *reinterpret_cast<float4*>(old[i]) = *reinterpret_cast<const float4*>(g);
        else
          old[i][0] = g[0];
      }
  }
  float acc[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
  bool from_before = key[1] == key[0];
#pragma unroll
  for (int i = 0; i < kTile; ++i)
    if (i < n && key[i + 1] < a.V) {
      v[i].add_to(acc);
      const bool last = key[i + 2] != key[i + 1];
      if (last || i == n - 1) {
        if (last && !from_before) {
          const int64_t at = int64_t(key[i + 1]) * a.d + c;
#pragma unroll
          for (int e = 0; e < VEC; ++e) acc[e] = ADD ? old[ADD ? i : 0][e] + acc[e] * a.scale : acc[e] * a.scale;
          if (ADD || a.grad_fp32)
            RowVec<float, VEC>::store(static_cast<float*>(a.grad) + at, acc);
          else
            RowVec<__nv_bfloat16, VEC>::store(static_cast<__nv_bfloat16*>(a.grad) + at, acc);
        } else {
          RowVec<float, VEC>::store(
              a.part + (int64_t(blockIdx.x) * 2 + (from_before ? 0 : 1)) * a.d + c, acc);
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
        from_before = false;
      }
    }
}

// Joins the partial sums of the runs that begin in one of the CTA's kJoinTiles
// tiles and end in a later one.  blockIdx.y: 32 * VEC columns.  A warp takes a
// tile and adds a short run's parts in order; a long run's are shared by the
// CTA's warps, every eighth part each, and the eight sums added in order.
constexpr int kJoinTiles = 8;
constexpr int kShortRun = 16;

template <int VEC, bool ADD>
__device__ __forceinline__ void finish_row(const SumArgs& a, int k, int64_t c, float (&s)[VEC]) {
  const int64_t at = int64_t(k) * a.d + c;
#pragma unroll
  for (int e = 0; e < VEC; ++e)
    s[e] = ADD ? static_cast<const float*>(a.grad)[at + e] + s[e] * a.scale : s[e] * a.scale;
  if (ADD || a.grad_fp32)
    RowVec<float, VEC>::store(static_cast<float*>(a.grad) + at, s);
  else
    RowVec<__nv_bfloat16, VEC>::store(static_cast<__nv_bfloat16*>(a.grad) + at, s);
}

template <int VEC, bool ADD>
__global__ void __launch_bounds__(32 * kJoinTiles) join_runs_kernel(SumArgs a, int64_t tiles) {
  __shared__ float acc[kJoinTiles][32][VEC];
  __shared__ int long_key[kJoinTiles];  // -1: no long run begins there
  __shared__ int64_t long_end[kJoinTiles];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t0 = int64_t(blockIdx.x) * kJoinTiles, t = t0 + warp, end = (t + 1) * kTile;
  const int64_t c = (int64_t(blockIdx.y) * 32 + lane) * VEC;
  int k = -1;
  int64_t last = t;  // the run's last tile
  if (end < a.N) {
    const int key = a.key[end - 1];
    const bool on = key < a.V && a.key[end] == key;
    const bool before = t > 0 && a.key[t * kTile] == key && a.key[t * kTile - 1] == key;
    if (on && !before) {
      k = key;
      for (;;) {  // 32 tiles a look
        const int64_t u = last + 1 + lane;
        const unsigned in = __ballot_sync(~0u, u < tiles && a.key[u * kTile] == k);
        last += in == ~0u ? 32 : __ffs(~in) - 1;
        if (in != ~0u) break;
      }
    }
  }
  const bool is_long = k >= 0 && last - t > kShortRun;
  if (lane == 0) {
    long_key[warp] = is_long ? k : -1;
    long_end[warp] = last;
  }
  if (k >= 0 && !is_long && c < a.d) {
    float s[VEC];
    RowVec<float, VEC>::load(a.part + (t * 2 + 1) * a.d + c, s);
#pragma unroll 8
    for (int64_t u = t + 1; u <= last; ++u) {
      float v[VEC];
      RowVec<float, VEC>::load(a.part + u * 2 * a.d + c, v);
#pragma unroll
      for (int e = 0; e < VEC; ++e) s[e] += v[e];
    }
    finish_row<VEC, ADD>(a, k, c, s);
  }
  __syncthreads();
  for (int i = 0; i < kJoinTiles; ++i) {
    if (long_key[i] < 0) continue;
    float s[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) s[e] = 0.f;
    if (c < a.d) {
      if (warp == 0) RowVec<float, VEC>::load(a.part + ((t0 + i) * 2 + 1) * a.d + c, s);
#pragma unroll 8
      for (int64_t u = t0 + i + 1 + warp; u <= long_end[i]; u += kJoinTiles) {
        float v[VEC];
        RowVec<float, VEC>::load(a.part + u * 2 * a.d + c, v);
#pragma unroll
        for (int e = 0; e < VEC; ++e) s[e] += v[e];
      }
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) acc[warp][lane][e] = s[e];
    __syncthreads();
    if (warp == 0 && c < a.d) {
#pragma unroll
      for (int g = 1; g < kJoinTiles; ++g)
#pragma unroll
        for (int e = 0; e < VEC; ++e) s[e] += acc[g][lane][e];
      finish_row<VEC, ADD>(a, long_key[i], c, s);
    }
    __syncthreads();
  }
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

template <int VEC, bool ADD>
cudaError_t run_sums(const LaunchEnv& env, const SumArgs& s, int64_t tiles) {
  const int64_t nv = s.d / VEC;
  const dim3 grid(unsigned(tiles), unsigned((nv + kSumThreads - 1) / kSumThreads));
  cudaError_t e = s.dy.fp32 ? launch_pdl(sum_rows_kernel<float, VEC, ADD>, grid, dim3(kSumThreads), 0,
                                         env.stream, s, int(nv))
                            : launch_pdl(sum_rows_kernel<__nv_bfloat16, VEC, ADD>, grid,
                                         dim3(kSumThreads), 0, env.stream, s, int(nv));
  if (e != cudaSuccess || tiles == 1) return e;
  return launch_pdl(join_runs_kernel<VEC, ADD>,
                    dim3(unsigned((tiles + kJoinTiles - 1) / kJoinTiles), unsigned((nv + 31) / 32)),
                    dim3(32 * kJoinTiles), 0, env.stream, s, tiles);
}

}  // namespace

cudaError_t launch_embed(const LaunchEnv& env, const EmbedArgs& a) {
  if (a.table_fp32)
    return a.out_fp32 ? run_embed<float, float>(env, a) : run_embed<float, __nv_bfloat16>(env, a);
  return a.out_fp32 ? run_embed<__nv_bfloat16, float>(env, a)
                    : run_embed<__nv_bfloat16, __nv_bfloat16>(env, a);
}

size_t embed_grad_scratch(int64_t N, int64_t d) {
  const size_t tiles = size_t((N + kTile - 1) / kTile);
  return 4 * up256(size_t(N) * 4) + up256(tiles * 2 * size_t(d) * 4);
}

cudaError_t launch_embed_grad(const LaunchEnv& env, const EmbedGradArgs& a) {
  const int64_t tiles = (a.N + kTile - 1) / kTile;
  const size_t col = up256(size_t(a.N) * 4);
  SortArgs so;
  so.ids = a.ids;
  so.ids64 = a.ids64;
  so.N = a.N;
  so.V = a.V;
  int bits = 1;
  while ((int64_t(1) << bits) <= a.V) ++bits;  // keys 0 .. V
  so.passes = (bits + kMaxBits - 1) / kMaxBits;
  so.bits = (bits + so.passes - 1) / so.passes;
  for (int i = 0; i < 2; ++i) {
    so.key[i] = reinterpret_cast<int*>(a.ws + i * col);
    so.pos[i] = reinterpret_cast<int*>(a.ws + (2 + i) * col);
  }
  const size_t table = size_t(a.V) * size_t(a.d) * (a.grad_fp32 ? 4 : 2);
  so.fill = a.accumulate ? nullptr : static_cast<uint4*>(a.grad);
  so.fill_vecs = a.accumulate ? 0 : int64_t(table / 16);
  so.fill_tail = a.accumulate ? 0 : int(table % 16);
  const size_t smem = (size_t(kSortWarps) * kBins + kBins + kSortWarps) * sizeof(int);
  cudaError_t e = cudaFuncSetAttribute(sort_ids_kernel,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
  if (e != cudaSuccess) return e;
  // the fill: up to two CTAs an SM, 16 vectors a thread at least
  int64_t fill = (so.fill_vecs + kSortThreads * 16 - 1) / (kSortThreads * 16);
  if (!a.accumulate) fill = std::max<int64_t>(fill, 1);
  fill = std::min<int64_t>(fill, 2 * env.num_sms);
  const int64_t ctas = kSortCtas + (fill + kSortCtas - 1) / kSortCtas * kSortCtas;
  e = launch_pdl(sort_ids_kernel, dim3(unsigned(ctas)), dim3(kSortThreads), smem, env.stream, so);
  if (e != cudaSuccess) return e;

  SumArgs s;
  s.key = so.key[(so.passes - 1) & 1];
  s.pos = so.pos[(so.passes - 1) & 1];
  s.N = a.N;
  s.V = a.V;
  s.d = a.d;
  s.dy = a.dy;
  s.scale = a.scale;
  s.grad = a.grad;
  s.grad_fp32 = a.grad_fp32;
  s.part = reinterpret_cast<float*>(a.ws + 4 * col);
  const bool vec = a.d % 8 == 0 && rows_aligned(a.dy.data, a.dy.stride_b, a.dy.stride_t, a.dy.fp32);
  if (a.accumulate) return vec ? run_sums<4, true>(env, s, tiles) : run_sums<1, true>(env, s, tiles);
  return vec ? run_sums<4, false>(env, s, tiles) : run_sums<1, false>(env, s, tiles);
}

}  // namespace ittt
