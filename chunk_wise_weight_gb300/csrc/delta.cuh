// delta.cuh -- what the gated delta rule's kernels share: warp-level matrix
// products whose operands are parts of fp32 numbers, and the tiles they read.
//
// Products with the state keep fp32 accuracy: an fp32 factor x is split into
// bf16 parts, hi = bf16(x), mid = bf16(x - hi), lo = bf16(x - hi - mid), 24
// bits together, and each part is multiplied on the tensor cores against the
// other factor, which is bf16 as given (q, k) or split the same way (then the
// products of parts p and r with p + r < 3 are kept).
//
// A walk is bound by the chain of dependent products from chunk to chunk, not by
// bytes or rates, and has two forms.  Calls of few heads use warp-level mma.sync on
// slices of 16 rows of dv, spread over the SMs: with the state transposed
// ([dv x dk]) the accumulators of each product are, register for register, the left
// operand of the next, where through tensor memory each link is a store, a fence, a
// commit and a load.  Calls of many heads use tcgen05 on whole heads, whose rate on
// 128 rows is four times as high.
#pragma once

#include "ops.h"
#include "rows.cuh"

namespace ittt {

// A lower triangular 64 x 64 bf16 image: its ten 16 x 16 blocks (i, j <= i),
// 512 bytes each, rows of 32 bytes whose two pieces are swapped in every other
// group of four rows (eight rows of one piece then cover all banks).
constexpr int kImage = 10 * 512;
__host__ __device__ constexpr int image_block(int i, int j) { return (i * (i + 1) / 2 + j) * 512; }
__device__ __forceinline__ int block_at(int r, int piece) {
  return r * 32 + ((piece ^ (r >> 2)) & 1) * 16;
}

// D (16 x 8, fp32) += A (16 x 16) B (16 x 8), bf16.
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void stsm4_t(uint32_t addr, uint32_t r0, uint32_t r1, uint32_t r2,
                                        uint32_t r3) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr),
               "r"(r0), "r"(r1), "r"(r2), "r"(r3)
               : "memory");
}

// 16 bytes global -> shared, zeros when !valid (nothing is read then).
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Splits two numbers into NP packed bf16 parts, each rounded to nearest (any
// number of leading parts is then the best sum of that many).
template <int NP>
__device__ __forceinline__ void split2(float x, float y, uint32_t (&p)[NP]) {
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    p[i] = pack_bf16x2(x, y);
    if (i + 1 < NP) {
      const float2 r = __ffma2_rn(
          make_float2(__uint_as_float(p[i] << 16), __uint_as_float(p[i] & 0xffff0000u)),
          make_float2(-1.f, -1.f), make_float2(x, y));
      x = r.x;
      y = r.y;
    }
  }
}

// The A operand (16 x 16) made of two accumulator tiles (16 x 8 each), in NP
// parts.
template <int NP>
__device__ __forceinline__ void split_frag(const float (&t0)[4], const float (&t1)[4],
                                           uint32_t (&a)[NP][4]) {
  uint32_t p[NP];
  split2<NP>(t0[0], t0[1], p);
#pragma unroll
  for (int i = 0; i < NP; ++i) a[i][0] = p[i];
  split2<NP>(t0[2], t0[3], p);
#pragma unroll
  for (int i = 0; i < NP; ++i) a[i][1] = p[i];
  split2<NP>(t1[0], t1[1], p);
#pragma unroll
  for (int i = 0; i < NP; ++i) a[i][2] = p[i];
  split2<NP>(t1[2], t1[3], p);
#pragma unroll
  for (int i = 0; i < NP; ++i) a[i][3] = p[i];
}

// Byte offset of 16-byte piece `c` of row `r` in a tile of CH (8 or 16)
// pieces a row; the swizzle spreads 8 rows of one piece over all banks.
template <int CH>
__device__ __forceinline__ uint32_t tile_at(int r, int c) {
  return uint32_t(r * CH + (c ^ (r & 7))) * 16;
}

// Lane addresses of the operand shapes below, for a tile of CH pieces a row.
// B operand, rows of the tile are the n index (tokens), columns the k index:
// registers 0, 1 for rows [8n, 8n+8), 2, 3 for [8n+8, 8n+16); k step s.
template <int CH>
__device__ __forceinline__ uint32_t addr_nk(int n, int s, int lane) {
  return tile_at<CH>(8 * (n + (lane >> 4)) + (lane & 7), 2 * s + ((lane >> 3) & 1));
}
// B operand, rows are the k index (step s), columns the n index: registers 0,
// 1 for columns [8n, 8n+8), 2, 3 for [8n+8, 8n+16).  Transposing load.
template <int CH>
__device__ __forceinline__ uint32_t addr_kn(int s, int n, int lane) {
  return tile_at<CH>(16 * s + (lane & 15), n + (lane >> 4));
}
// A operand, rows [16m, 16m+16) of the tile, columns k step s.
template <int CH>
__device__ __forceinline__ uint32_t addr_mk(int m, int s, int lane) {
  return tile_at<CH>(16 * m + (lane & 15), 2 * s + (lane >> 4));
}
// The same out of one block of an image: B operand with rows the n index ...
__device__ __forceinline__ uint32_t block_nk(int lane) {
  return block_at(8 * (lane >> 4) + (lane & 7), (lane >> 3) & 1);
}
// ... with rows the k index (transposing load) ...
__device__ __forceinline__ uint32_t block_kn(int lane) { return block_at(lane & 15, lane >> 4); }
// ... and A operand whose rows are the block's columns (transposing load).
__device__ __forceinline__ uint32_t block_km(int lane) {
  return block_at(8 * (lane >> 4) + (lane & 7), (lane >> 3) & 1);
}

// Loads a [64 x dim] bf16 tile (CH pieces a row, swizzled) of `n` rows, zeros
// below; all threads of the CTA, completed by cp_wait + barrier.
__device__ __forceinline__ void store_piece(unsigned char* dst, const __nv_bfloat16* src) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = __bfloat16_as_ushort(src[2 * i]), hi = __bfloat16_as_ushort(src[2 * i + 1]);
    w[i] = lo | (hi << 16);
  }
  *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
}

template <int CH>
__device__ __forceinline__ void load_tile(unsigned char* dst, const __nv_bfloat16* src, int64_t st,
                                          int n, bool vec, int tid, int threads) {
  for (int i = tid; i < kDeltaChunk * CH; i += threads) {
    const int r = i / CH, c = i % CH;
    unsigned char* d = dst + tile_at<CH>(r, c);
    const __nv_bfloat16* s = src + (r < n ? r * st : 0) + c * 8;
    if (vec)
      cp16(smem_u32(d), s, r < n);
    else if (r < n)
      store_piece(d, s);
    else
      *reinterpret_cast<uint4*>(d) = make_uint4(0, 0, 0, 0);
  }
}

// The same for `pieces` columns of 8 with rows of (pieces + 1) * 16 bytes
// (an odd multiple of 16 when pieces is even: no bank conflicts).
__device__ __forceinline__ void load_cols(unsigned char* dst, const __nv_bfloat16* src, int64_t st,
                                          int pieces, int n, bool vec, int tid, int threads) {
  const int pitch = (pieces + 1) * 16;
  for (int i = tid; i < kDeltaChunk * pieces; i += threads) {
    const int r = i / pieces, c = i - r * pieces;
    unsigned char* d = dst + r * pitch + c * 16;
    const __nv_bfloat16* s = src + (r < n ? r * st : 0) + c * 8;
    if (vec)
      cp16(smem_u32(d), s, r < n);
    else if (r < n)
      store_piece(d, s);
    else
      *reinterpret_cast<uint4*>(d) = make_uint4(0, 0, 0, 0);
  }
}

// Sum of two floats kept as a pair, so that differences of running sums keep
// their low bits: a gate of -1000 does not blur its neighbours' decays.
struct Pair {
  float hi, lo;
};
__device__ __forceinline__ float decay(const Pair& i, const Pair& j) {
  return expf((i.hi - j.hi) + (i.lo - j.lo));
}

// Running sums G of the gates of the 64 tokens from (b, t) of head h, by one
// warp: in double, two a lane, then across lanes.  A decay of e^-1000 is zero
// in fp32, so lower gates count as -1000 (minus infinity, a full reset, among
// them).
__device__ __forceinline__ void gate_sums(const GateView& gv, int64_t b, int64_t t, int h, int n,
                                          int lane, Pair* G) {
  double x[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = 2 * lane + i;
    const float g = r < n ? gv.data[b * gv.sb + (t + r) * gv.st + h * gv.sh] : 0.f;
    x[i] = g < -1000.f ? -1000.0 : double(g);
  }
  x[1] += x[0];
  double sum = x[1];
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const double v = __shfl_up_sync(~0u, sum, m);
    if (lane >= m) sum += v;
  }
  const double before = sum - x[1];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const double v = before + x[i];
    G[2 * lane + i].hi = float(v);
    G[2 * lane + i].lo = float(v - double(float(v)));
  }
}

// What the first kernel leaves for each (chunk, head), in bytes:
//   E map   (I + B diag(beta))^-1, B_ij = e^{G_i - G_j} k_i.k_j (j < i): 3 parts
//   scores  scale e^{G_i - G_j} q_i.k_j (j <= i): 3 parts
//   gates   e^{G_i}, e^{G_63 - G_i}, beta_i: fp32 [3][64]
//   (gradient only)  R map  (I + diag(beta) B)^-1: 3 parts
// each part an image.
constexpr int kBlkE = 0;
constexpr int kBlkM = 3 * kImage;
constexpr int kBlkGate = 6 * kImage;
constexpr int kBlkFwd = kBlkGate + 1024;
constexpr int kBlkR = kBlkFwd;
constexpr int kBlkGrad = kBlkFwd + 3 * kImage;

// ------------------------------------------------------------ links of the walk
// Both walks carry 16 rows of a state ([dv x dk], fp32), a slice, in the
// accumulator registers of a team of four warps, one on each scheduler: warp w
// holds a quarter of the dk columns, and of every product with tokens as
// columns it takes tokens [16w, 16w + 16) of the chunk.  A chunk is three links,
//   P = state K^T, Y = X map^T (X made of P), state = last state + W K (W of Y),
// and before each link the warps hand one another its left operand, split into
// three parts, through shared memory.  One warp alone spends twice the tensor
// cores' time on a chunk (its arithmetic between products cannot overlap them);
// four share both.  The right operands of a link are loaded before the barrier
// ahead of it.
//
// The products of a sum go to one accumulator for each part of the left
// operand: the tensor cores round sums towards zero, so additions at full size
// are kept few, and the chains of dependent products short.
constexpr int kTeam = 128;
constexpr int kOperand = 512;  // one part of an operand: 32 lanes x 16 bytes

__device__ __forceinline__ void team_bar(int slice) {
  asm volatile("bar.sync %0, 128;" ::"r"(1 + slice) : "memory");
}

template <int N>
__device__ __forceinline__ void zero(float (&t)[N][4]) {
#pragma unroll
  for (int j = 0; j < N; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) t[j][e] = 0.f;
}

// Two tiles (16 x 8 each) += a b.
__device__ __forceinline__ void mma2(float (&d0)[4], float (&d1)[4], const uint32_t (&a)[4],
                                     const uint32_t (&b)[4]) {
  mma16816(d0, a, b[0], b[1]);
  mma16816(d1, a, b[2], b[3]);
}

__device__ __forceinline__ void put_operand(unsigned char* to, const uint32_t (&a)[4], int lane) {
  *reinterpret_cast<uint4*>(to + lane * 16) = make_uint4(a[0], a[1], a[2], a[3]);
}
__device__ __forceinline__ void get_operand(uint32_t (&a)[4], const unsigned char* from, int lane) {
  const uint4 v = *reinterpret_cast<const uint4*>(from + lane * 16);
  a[0] = v.x;
  a[1] = v.y;
  a[2] = v.z;
  a[3] = v.w;
}
// Splits a pair of tiles into NP parts and hands them over as step ks.
template <int NP>
__device__ __forceinline__ void put_tiles(unsigned char* to, int ks, const float (&t0)[4],
                                          const float (&t1)[4], int lane) {
  uint32_t a[NP][4];
  split_frag<NP>(t0, t1, a);
#pragma unroll
  for (int p = 0; p < NP; ++p) put_operand(to + (ks * NP + p) * kOperand, a[p], lane);
}
// A state as the gradient's last kernel reads it, three parts: for each panel of 64
// rows of dv (the last may be shorter) and each part, pieces of 8 columns of dk, each
// [rows][16 bytes].  Neighbouring rows are neighbours in memory (a warp whose lanes
// are rows stores without gaps), and eight rows of a piece are a core matrix of an
// operand without swizzle.
constexpr int kPanel = 64;
__host__ __device__ constexpr int64_t state_parts(int dv, int dk) { return int64_t(3) * dv * dk * 2; }
template <int DK>
__device__ __forceinline__ int64_t piece_at(int dv, int row, int part, int piece) {
  const int panel = row / kPanel, rows = min(kPanel, dv - panel * kPanel);
  return int64_t(panel) * 3 * kPanel * DK * 2 + (int64_t(part) * (DK / 8) + piece) * rows * 16 + (row % kPanel) * 16;
}

// This warp's columns of the state, as the left operand of the next chunk.  SNAP:
// its parts also go to `snap` (unless null); `row` is the slice's first row.
template <int DK, bool SNAP>
__device__ __forceinline__ void put_state(unsigned char* to, const float (&S)[DK / 32][4], int w, int lane,
                                          unsigned char* snap = nullptr, int row = 0, int dv = 0) {
#pragma unroll
  for (int ks = 0; ks < DK / 64; ++ks) {
    const int step = w * (DK / 64) + ks;
    uint32_t a[3][4];
    split_frag<3>(S[2 * ks], S[2 * ks + 1], a);
#pragma unroll
    for (int p = 0; p < 3; ++p) put_operand(to + (step * 3 + p) * kOperand, a[p], lane);
    if (SNAP && snap != nullptr) {
#pragma unroll
      for (int p = 0; p < 3; ++p)
#pragma unroll
        for (int half = 0; half < 2; ++half) {  // a[.][e]: rows + 8 (e & 1), pieces + (e >> 1)
          unsigned char* at = snap + piece_at<DK>(dv, row + (lane >> 2), p, 2 * step + half) + 4 * (lane & 3);
          *reinterpret_cast<uint32_t*>(at) = a[p][2 * half];
          *reinterpret_cast<uint32_t*>(at + 128) = a[p][2 * half + 1];
        }
    }
  }
}

template <int NP>
__device__ __forceinline__ void sum_parts(const float (&t)[NP][2][4], float (&to)[2][4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float x = t[NP - 1][i][e];
#pragma unroll
      for (int p = NP - 2; p >= 0; --p) x += t[p][i][e];
      to[i][e] = x;
    }
}

// This warp's 16 tokens of (K S^T)^T and, from the first NQ parts of the state,
// of (Q S^T)^T; the state's operands at `sop`, [DK / 16][3][kOperand].
template <int DK, int NQ>
__device__ __forceinline__ void state_times_rows(const unsigned char* sop, uint32_t sk, uint32_t sq, int w,
                                                 int lane, float (&P)[2][4], float (&O)[2][4]) {
  float tp[3][2][4], tq[NQ ? NQ : 1][2][4];
#pragma unroll
  for (int p = 0; p < 3; ++p) zero(tp[p]);
#pragma unroll
  for (int p = 0; p < NQ; ++p) zero(tq[p]);
#pragma unroll
  for (int ks = 0; ks < DK / 16; ++ks) {
    uint32_t bk[4], bq[4], sa[3][4];
    ldsm4(bk, sk + addr_nk<DK / 8>(2 * w, ks, lane));
    if (NQ) ldsm4(bq, sq + addr_nk<DK / 8>(2 * w, ks, lane));
#pragma unroll
    for (int p = 0; p < 3; ++p) get_operand(sa[p], sop + (ks * 3 + p) * kOperand, lane);
#pragma unroll
    for (int p = 0; p < 3; ++p) mma2(tp[p][0], tp[p][1], sa[p], bk);
#pragma unroll
    for (int p = 0; p < NQ; ++p) mma2(tq[p][0], tq[p][1], sa[p], bq);
  }
  sum_parts<3>(tp, P);
  if constexpr (NQ > 0) sum_parts<NQ>(tq, O);
}

// The blocks of a triangular image that this warp's tokens meet, NP parts of
// it, as right operands: X map^T (TRANS: X map) for tokens [16w, 16w + 16).
template <bool TRANS, int NP>
__device__ __forceinline__ void load_map(uint32_t (&b)[4][NP][4], uint32_t map, int w, int lane) {
#pragma unroll
  for (int ks = 0; ks < 4; ++ks)
    if (TRANS ? ks >= w : ks <= w)
#pragma unroll
      for (int r = 0; r < NP; ++r) {
        if (TRANS)
          ldsm4_t(b[ks][r], map + r * kImage + image_block(ks, 0) + w * 512 + block_kn(lane));
        else
          ldsm4(b[ks][r], map + r * kImage + image_block(w, 0) + ks * 512 + block_nk(lane));
      }
}

// Y = this warp's 16 tokens of X map^T (TRANS: X map), from the operands of X,
// [4][NP][kOperand].
template <bool TRANS, int NP>
__device__ __forceinline__ void map_tokens(const unsigned char* x, const uint32_t (&b)[4][NP][4], int w,
                                           int lane, float (&Y)[2][4]) {
  float t[NP][2][4];  // by p + r
#pragma unroll
  for (int p = 0; p < NP; ++p) zero(t[p]);
#pragma unroll
  for (int ks = 0; ks < 4; ++ks)
    if (TRANS ? ks >= w : ks <= w) {
      uint32_t xa[NP][4];
#pragma unroll
      for (int p = 0; p < NP; ++p) get_operand(xa[p], x + (ks * NP + p) * kOperand, lane);
#pragma unroll
      for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int r = 0; p + r < NP; ++r) mma2(t[p + r][0], t[p + r][1], xa[p], b[ks][r]);
    }
  sum_parts<NP>(t, Y);
}

// Y += this warp's 16 tokens of X map^T, with the map's blocks read as they are met
// (off the chain: held from before a barrier they would only cost registers).
__device__ __forceinline__ void add_map_tokens(const unsigned char* x, uint32_t map, int w, int lane, float (&Y)[2][4]) {
  float t[3][2][4];  // by p + r
#pragma unroll
  for (int p = 0; p < 3; ++p) zero(t[p]);
#pragma unroll
  for (int ks = 0; ks < 4; ++ks)
    if (ks <= w) {
      uint32_t xa[3][4], b[3][4];
#pragma unroll
      for (int r = 0; r < 3; ++r) ldsm4(b[r], map + r * kImage + image_block(w, 0) + ks * 512 + block_nk(lane));
#pragma unroll
      for (int p = 0; p < 3; ++p) get_operand(xa[p], x + (ks * 3 + p) * kOperand, lane);
#pragma unroll
      for (int p = 0; p < 3; ++p)
#pragma unroll
        for (int r = 0; p + r < 3; ++r) mma2(t[p + r][0], t[p + r][1], xa[p], b[r]);
    }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) Y[i][e] += t[0][i][e] + (t[1][i][e] + t[2][i][e]);
}

// This warp's dk columns of the rows of a tile, as right operands of W rows.
template <int DK>
__device__ __forceinline__ void load_rows(uint32_t (&b)[4][DK / 64][4], uint32_t rows, int w, int lane) {
#pragma unroll
  for (int ks = 0; ks < 4; ++ks)
#pragma unroll
    for (int j = 0; j < DK / 64; ++j)
      ldsm4_t(b[ks][j], rows + addr_kn<DK / 8>(ks, w * (DK / 32) + 2 * j, lane));
}
// acc = W rows, from the operands of W, [4][3][kOperand].
template <int DK>
__device__ __forceinline__ void outer_rows(float (&acc)[DK / 32][4], const unsigned char* wop,
                                           const uint32_t (&b)[4][DK / 64][4], int lane) {
  uint32_t wa[4][3][4];
#pragma unroll
  for (int ks = 0; ks < 4; ++ks)
#pragma unroll
    for (int p = 0; p < 3; ++p) get_operand(wa[ks][p], wop + (ks * 3 + p) * kOperand, lane);
  zero(acc);
#pragma unroll
  for (int p = 2; p >= 0; --p)
#pragma unroll
    for (int ks = 0; ks < 4; ++ks)
#pragma unroll
      for (int j = 0; j < DK / 64; ++j) mma2(acc[2 * j], acc[2 * j + 1], wa[ks][p], b[ks][j]);
}

// The two stages of a walk and who fills them: a warp of its own, cp.async for
// K, Q and the columns, one bulk copy for the chunk's block (its completion
// counted by a barrier that every thread then waits on).
struct StageBars {
  uint64_t full[2];
  int abort;
};
__device__ __forceinline__ void init_bars(StageBars* bars) {
  if (threadIdx.x == 0) {
    mbar_init(&bars->full[0], 1);
    mbar_init(&bars->full[1], 1);
    bars->abort = 0;
    fence_mbar_init();
  }
  __syncthreads();
}
// Whether the wait has run out: the CTA then stops at the chunk's next barrier, all
// roles together, before another copy is issued.
__device__ __forceinline__ bool wait_block(StageBars* bars, int it, unsigned int* status) {
  const bool late = !mbar_wait(&bars->full[it & 1], (it >> 1) & 1, &bars->abort);
  if (late) raise_abort(&bars->abort, status, kStatusTimeout);
  return late;
}

// A [64 x dim] tile by one warp: 16-byte pieces, rows of the tile `st` elements
// apart in memory; pieces from `cols` on are zero.
template <int CH>
__device__ __forceinline__ void warp_load_tile(unsigned char* dst, const __nv_bfloat16* src, int64_t st,
                                               int n, bool vec, int lane, int cols = CH) {
  constexpr int RP = 32 / CH;  // rows side by side
  const int c = lane % CH, r0 = lane / CH;
  if (c >= cols) n = 0;
  const __nv_bfloat16* p = src + r0 * st + c * 8;
  if (vec) {
    const uint32_t d = smem_u32(dst);
#pragma unroll 8
    for (int r = r0; r < kDeltaChunk; r += RP, p += RP * st) cp16(d + tile_at<CH>(r, c), r < n ? p : src, r < n);
  } else {
    for (int r = r0; r < kDeltaChunk; r += RP, p += RP * st) {
      unsigned char* d = dst + tile_at<CH>(r, c);
      if (r < n)
        store_piece(d, p);
      else
        *reinterpret_cast<uint4*>(d) = make_uint4(0, 0, 0, 0);
    }
  }
}

// A warp's quarter of a slice of a state: 16 rows from `row`, DK / 4 columns.
template <int DK>
__device__ __forceinline__ void load_state(float (&S)[DK / 32][4], const float* from, int64_t row, int w,
                                           int lane) {
#pragma unroll
  for (int j = 0; j < DK / 32; ++j) {
    float2 lo = make_float2(0.f, 0.f), hi = lo;
    if (from) {
      const float* p = from + (row + (lane >> 2)) * DK + w * (DK / 4) + 8 * j + 2 * (lane & 3);
      lo = *reinterpret_cast<const float2*>(p);
      hi = *reinterpret_cast<const float2*>(p + 8 * DK);
    }
    S[j][0] = lo.x;
    S[j][1] = lo.y;
    S[j][2] = hi.x;
    S[j][3] = hi.y;
  }
}
template <int DK>
__device__ __forceinline__ void store_state(const float (&S)[DK / 32][4], float* to, int64_t row, int w,
                                            int lane) {
  float* p = to + (row + (lane >> 2)) * DK + w * (DK / 4) + 2 * (lane & 3);
#pragma unroll
  for (int j = 0; j < DK / 32; ++j) {
    *reinterpret_cast<float2*>(p + 8 * j) = make_float2(S[j][0], S[j][1]);
    *reinterpret_cast<float2*>(p + 8 * DK + 8 * j) = make_float2(S[j][2], S[j][3]);
  }
}

// A warp's [16 dv x 16 tokens] to rows of a [token][..] bf16 array: the first
// `n` tokens, `stride` elements apart, through 512 bytes at `box`.
__device__ __forceinline__ void store_tokens(const float (&T)[2][4], unsigned char* box,
                                             __nv_bfloat16* to, int64_t stride, int n, int lane) {
  stsm4_t(smem_u32(box) + (8 * (lane >> 4) + (lane & 7)) * 32 + ((lane >> 3) & 1) * 16,
          pack_bf16x2(T[0][0], T[0][1]), pack_bf16x2(T[0][2], T[0][3]), pack_bf16x2(T[1][0], T[1][1]),
          pack_bf16x2(T[1][2], T[1][3]));
  __syncwarp();
  const int r = lane >> 1, half = lane & 1;
  if (r < n)
    *reinterpret_cast<uint4*>(to + r * stride + 8 * half) =
        *reinterpret_cast<const uint4*>(box + r * 32 + half * 16);
}

// A warp's [16 dv x 16 tokens] into the tile of its rows: [3 parts][dv][64 tokens],
// 128-byte rows with swizzled pieces.
__device__ __forceinline__ void store_token_parts(const float (&T)[2][4], unsigned char* to, int dv, int row, int w,
                                                  int lane) {
  uint32_t a[3][4];
  split_frag<3>(T[0], T[1], a);
  const int r = row + (lane >> 2);
  unsigned char* at = to + int64_t(r) * 128 + 4 * (lane & 3);
#pragma unroll
  for (int p = 0; p < 3; ++p)
#pragma unroll
    for (int e = 0; e < 4; ++e)  // rows + 8 (e & 1), pieces + (e >> 1)
      *reinterpret_cast<uint32_t*>(at + int64_t(p) * dv * 128 + (e & 1) * 1024 +
                                   (((2 * w + (e >> 1)) ^ (r & 7)) << 4)) = a[p][e];
}

// A warp's 16 tokens of a [64 tokens][16 dv] column block, transposed: v[2i],
// v[2i + 1] hold tile i's rows lane / 4 and lane / 4 + 8 of dv.
__device__ __forceinline__ void load_cols_t(uint32_t (&v)[4], uint32_t cols, int pitch, int w, int lane) {
  ldsm4_t(v, cols + (8 * (2 * w + (lane >> 4)) + (lane & 7)) * pitch + ((lane >> 3) & 1) * 16);
}

// Sums of 16 numbers over the lanes of a warp; lanes 0, 2, .. 30 store them.
__device__ __forceinline__ void store_row_sums(float (&x)[16], float* to, int lane) {
  int m = 16;
#pragma unroll
  for (int cnt = 8; cnt >= 1; cnt >>= 1, m >>= 1) {
    const bool up = lane & m;
#pragma unroll
    for (int i = 0; i < cnt; ++i) {
      const float send = up ? x[i] : x[i + cnt], keep = up ? x[i + cnt] : x[i];
      x[i] = keep + __shfl_xor_sync(~0u, send, m);
    }
  }
  x[0] += __shfl_xor_sync(~0u, x[0], 1);
  if ((lane & 1) == 0) to[lane >> 1] = x[0];
}
// Slices a CTA of a walk: one while every slice has an SM of its own, two beyond
// that, which share the loads of K, Q and the chunk's block and fill each other's
// waits.  1024 tokens, heads of 128 x 128, one / two slices a CTA: 16 heads (128
// slices) 55 / 74 us, gradient 160 / 188; 20 heads (160) 98 / 74 us, 234 / 210.
inline int walk_slices(int ndocs, int Hv, int dv, int num_sms) {
  return dv % 32 == 0 && int64_t(ndocs) * Hv * (dv / 16) > num_sms ? 2 : 1;
}

// The blocks as the walks read them: each part a tile of 64 rows of 128 bytes,
// swizzled (blocks above the diagonal are not written, and not read).
constexpr int kWideTile = 8192;
constexpr int kWideM = 3 * kWideTile;
constexpr int kWideGate = 6 * kWideTile;
constexpr int kWideFwd = kWideGate + 1024;
constexpr int kWideR = kWideFwd;
constexpr int kWideGrad = kWideR + 3 * kWideTile;

// Fills those blocks for every chunk and head (wide: as tiles).
cudaError_t launch_delta_prepare(const LaunchEnv& env, const DeltaArgs& a, unsigned char* blocks,
                                 bool grad, bool wide);

// What the gradient's forward walk keeps.
struct DeltaSave {
  unsigned char* snap;  // [nchunks][Hv]: the state at the chunk's start
  unsigned char* e;     // [nchunks][Hv][3 parts][dv][64]: E, transposed (see store_token_parts)
};
__host__ __device__ constexpr int64_t token_tiles(int dv) { return int64_t(dv) * 3 * 128; }

// The gradient's reverse walk.
struct ReverseArgs {
  HeadView q, k, dout;
  int Hk, Hv, dv, T;
  DeltaMap map;
  float scale;
  const unsigned char* blocks;
  unsigned int* status;
  const float* dstate_out;
  float* dstate_in;
  __nv_bfloat16* dvp;
  unsigned char* dr;     // dR, laid out as E
  unsigned char* dsnap;  // [nchunks][Hv]: dS' of each chunk
};

// Whether the walks (forward; forward for the gradient; reverse) give an SM a whole
// head rather than slices of 16 rows.
bool delta_by_head(int64_t sequences, int Hv, int dv, int num_sms);

cudaError_t launch_team_walk(const LaunchEnv& env, const DeltaArgs& a, const unsigned char* blocks,
                             const DeltaSave* save);
cudaError_t launch_head_walk(const LaunchEnv& env, const DeltaArgs& a, const unsigned char* blocks,
                             const DeltaSave* save);
cudaError_t launch_head_reverse(const LaunchEnv& env, const ReverseArgs& r, int dk);

// ------------------------------------------------------- tcgen05, by a warp
// One lane of a converged warp.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t on;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(on));
  return on;
}

// D[tmem] (+)= A[smem] * B[smem]^T, issued by the elected lane of a warp whose
// lanes all hold the same arguments: they then stay in uniform registers (issued
// from a branch of one lane, each product cost its issuer 60 to 100 cycles, twice
// what the product itself takes).  `a_lo`, `b_lo`: the low words of descriptors
// (128-byte rows, swizzled, groups of eight rows 1024 bytes apart; `b_hi`: another
// form of B).
__device__ __forceinline__ void mma_ss(uint32_t elected, uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo,
                                       uint32_t idesc, uint32_t accumulate,
                                       uint32_t b_hi = (1024u >> 4) | (1u << 14) | (2u << 29)) {
  constexpr uint32_t kHi = (1024u >> 4) | (1u << 14) | (2u << 29);
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 da, db;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "setp.ne.b32 q, %6, 0;\n\t"
      "mov.b64 da, {%1, %3};\n\t"
      "mov.b64 db, {%2, %7};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(kHi), "r"(idesc), "r"(accumulate), "r"(elected), "r"(b_hi)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t elected, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(elected)
      : "memory");
}

// 16 fp32 columns of this thread's row.
__device__ __forceinline__ void read16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    asm volatile("" : "+r"(r[i]));  // not before the wait
    v[i] = __uint_as_float(r[i]);
  }
}

}  // namespace ittt
