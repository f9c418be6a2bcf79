// k_delta_grad.cu -- gradients of the gated delta rule, in chunks of 64 tokens.
//
// With the chunk's forward quantities (S the state at its start, S' at its
// end, E, U = b E, the scores M, D_ij = e^{G_i - G_j}; see k_delta.cu) and the
// gradient dS' that comes from the chunks after it:
//   dU0 = M^T dO + e^{G_63 - G} (K dS'^T)
//   dR  = (I + diag(b) B)^-T dU0             gradient at b X
//   dV  = b dR =: dX,   db_i = dR_i.E_i
//   dS  = e^{G_63} dS' + scale (e^G dO)^T Q - (e^G dX)^T K
//   dq_i = scale e^{G_i} dO_i S + sum_{j <= i} scale D_ij (dO_i.U_j) k_j
//   dk_j = sum_{i >= j} scale D_ij (dO_i.U_j) q_i - e^{G_j} dX_j S + e^{G_63 - G_j} U_j dS'
//          - sum_{i < j} D_ji (dX_j.U_i) k_i - sum_{i > j} D_ij (dX_i.U_j) k_i
//   dg_t = sum_{i >= t} a_i + sum_{i >= t > j} B_ij + sum_{j < t} c_j + e^{G_63} <dS', S>
//          a_i = scale e^{G_i} dO_i S.q_i - e^{G_i} dX_i S.k_i
//          B_ij = scale D_ij (dO_i.U_j) (q_i.k_j) - D_ij (dX_i.U_j) (k_i.k_j)
//          c_j = e^{G_63 - G_j} U_j dS'.k_j
// (dg_t gathers every decay that spans token t.  Each term carries its own decay and
// none is subtracted from another, so dg is as exact in a head that forgets within a
// token as in one that keeps thousands, and zero at a reset.  The sums telescope to
// products of dO with O and dV with V, which cancel: at g = -12 a tenth of dg was lost.)
//
// Four kernels: the chunks' blocks and the forward walk (k_delta.cu) keep S and E; a
// reverse walk, of the same shape, carries dS and leaves dR and dS'; then everything
// else, of every chunk at once.  2 x 4096 tokens, 20 heads of 128 x 128: 95 + 277 + 338 +
// 311 us; bound by the two walks' chains and by the last kernel's passes, whose products
// and sums take turns.
#include <algorithm>

#include "delta.cuh"

namespace ittt {
namespace {

// Shared memory of a CTA of `ns` slices: two stages (K, Q, scores, gates, R map, dO),
// then what each slice's warps exchange.
template <int DK>
struct ReverseShape {
  static constexpr int kTile = kDeltaChunk * DK * 2;
  static constexpr int kBlk = kBlkGrad - kBlkM;  // scores, gates, R map
  static constexpr int kGate = 2 * kTile + kBlkGate - kBlkM;
  static constexpr int kR = 2 * kTile + kBlkR - kBlkM;
  static constexpr int kCols = 2 * kTile + kBlk;
  static constexpr int kX = DK / 16 * 3 * kOperand;  // operands of dU0, after those of dS'
  static constexpr int kW = kX + 12 * kOperand;      // of -e^G dX
  static constexpr int kY = kW + 12 * kOperand;      // of scale e^G dO
  static constexpr int kOwn = kY + 12 * kOperand;
  static __host__ __device__ constexpr int stage(int ns) {
    return kCols + kDeltaChunk * (2 * ns + 1) * 16;
  }
  static __host__ __device__ constexpr int smem(int ns) {
    return 2 * stage(ns) + ns * kOwn + int(sizeof(StageBars));
  }
};

// The forward walk's shape, from the last chunk to the first, with dS in place
// of the state.
template <int DK>
__global__ void __launch_bounds__(2 * kTeam + 32) delta_reverse_kernel(ReverseArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  using W = ReverseShape<DK>;
  const int ns = blockDim.x / kTeam, tid = threadIdx.x, lane = tid & 31, slice = tid / kTeam;
  const int w = slice & 1 ? 3 - ((tid >> 5) & 3) : (tid >> 5) & 3;
  const int pieces = 2 * ns, pitch = (pieces + 1) * 16;
  const int stage_bytes = W::stage(ns);
  const int parts = a.dv / (16 * ns);
  const int h = (blockIdx.x / parts) % a.Hv, s = blockIdx.x / (parts * a.Hv);
  const int col0 = (blockIdx.x % parts) * 16 * ns, row0 = col0 + 16 * slice;
  const int t2 = 2 * (lane & 3);
  unsigned char* own = smem + 2 * stage_bytes + slice * W::kOwn;
  StageBars* bars = reinterpret_cast<StageBars*>(smem + 2 * stage_bytes + ns * W::kOwn);
  init_bars(bars);
  griddep_wait();
  griddep_launch_dependents();
  const int64_t b = a.map.row(s), tok0 = a.map.start(s);
  const int len = a.map.len(s), nchunks = (len + kDeltaChunk - 1) / kDeltaChunk;
  const int64_t chunk0 = a.map.chunk0(s);

  if (slice == ns) {  // the loader
    const int hk = h / (a.Hv / a.Hk);
    const auto* kp = static_cast<const __nv_bfloat16*>(a.k.data) + b * a.k.sb + tok0 * a.k.st + hk * a.k.sh;
    const auto* qp = static_cast<const __nv_bfloat16*>(a.q.data) + b * a.q.sb + tok0 * a.q.st + hk * a.q.sh;
    const auto* dop = static_cast<const __nv_bfloat16*>(a.dout.data) + b * a.dout.sb + tok0 * a.dout.st + h * a.dout.sh + col0;
    for (int it = 0; it <= nchunks; ++it) {
      if (it < nchunks) {
        const int c = nchunks - 1 - it;
        unsigned char* st = smem + (it & 1) * stage_bytes;
        const int n = min(kDeltaChunk, len - c * kDeltaChunk);
        const int64_t t = int64_t(c) * kDeltaChunk;
        if (lane == 0) {
          mbar_arrive_expect_tx(&bars->full[it & 1], W::kBlk);
          bulk_load(st + 2 * W::kTile, a.blocks + ((chunk0 + c) * a.Hv + h) * int64_t(kBlkGrad) + kBlkM, W::kBlk,
                    &bars->full[it & 1]);
        }
        warp_load_tile<DK / 8>(st, kp + t * a.k.st, a.k.st, n, a.k.vec, lane);
        warp_load_tile<DK / 8>(st + W::kTile, qp + t * a.q.st, a.q.st, n, a.q.vec, lane);
        load_cols(st + W::kCols, dop + t * a.dout.st, a.dout.st, pieces, n, a.dout.vec, lane, 32);
        cp_wait_all();
      }
      if (__syncthreads_or(0)) break;
    }
    settle(&bars->abort);
    return;
  }

  float S[DK / 32][4];  // dS'
  const int64_t srow = (int64_t(s) * a.Hv + h) * a.dv + row0;
  load_state<DK>(S, a.dstate_out, srow, w, lane);
  auto snapshot = [&](int c) {
    return c < 0 ? nullptr : a.dsnap + ((chunk0 + c) * a.Hv + h) * state_parts(a.dv, DK);
  };
  put_state<DK, true>(own, S, w, lane, snapshot(nchunks - 1), row0, a.dv);
  bool late = false;
  for (int it = 0;; ++it) {
    if (__syncthreads_or(late) || it == nchunks) break;
    const int c = nchunks - 1 - it;
    late = wait_block(bars, it, a.status);
    const unsigned char* st = smem + (it & 1) * stage_bytes;
    const uint32_t sk = smem_u32(st), sq = sk + W::kTile;
    const uint32_t sd = sk + W::kCols + 32 * slice;
    const float* gate = reinterpret_cast<const float*>(st + W::kGate) + 16 * w + t2;  // this warp's tokens
    const int64_t ch = (chunk0 + c) * a.Hv + h;
    float X[2][4];
    {
      float none[2][4];
      state_times_rows<DK, 0>(own, sk, 0, w, lane, X, none);
    }
    {
      // this warp's step of scale e^G dO, as an operand
      uint32_t v[4];
      float y[2][4];
      load_cols_t(v, sd, pitch, w, lane);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 eg = *reinterpret_cast<const float2*>(gate + 8 * i);
        const float2 d0 = unpack_bf16x2(v[2 * i]), d1 = unpack_bf16x2(v[2 * i + 1]);
        y[i][0] = a.scale * eg.x * d0.x;
        y[i][1] = a.scale * eg.y * d0.y;
        y[i][2] = a.scale * eg.x * d1.x;
        y[i][3] = a.scale * eg.y * d1.y;
      }
      put_tiles<3>(own + W::kY, w, y[0], y[1], lane);
    }
    {
      // dU0 = e^{G_63 - G} (K dS'^T) + M^T dO, this warp's tokens
      uint32_t bm[4][3][4];
      float t[3][2][4], D[2][4];
      load_map<true, 3>(bm, sk + 2 * W::kTile, w, lane);
#pragma unroll
      for (int r = 0; r < 3; ++r) zero(t[r]);
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
        if (ks >= w) {
          uint32_t dO[4];  // left operand: 16 rows of dv, 16 tokens
          load_cols_t(dO, sd, pitch, ks, lane);
#pragma unroll
          for (int r = 0; r < 3; ++r) mma2(t[r][0], t[r][1], dO, bm[ks][r]);
        }
      sum_parts<3>(t, D);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 ge = *reinterpret_cast<const float2*>(gate + 64 + 8 * i);
#pragma unroll
        for (int e = 0; e < 4; ++e) X[i][e] = (e & 1 ? ge.y : ge.x) * X[i][e] + D[i][e];
      }
      put_tiles<3>(own + W::kX, w, X[0], X[1], lane);
    }
    float R[2][4];
    {
      uint32_t br[4][3][4];
      load_map<true, 3>(br, sk + W::kR, w, lane);
      team_bar(slice);
      map_tokens<true, 3>(own + W::kX, br, w, lane, R);  // dR
    }
    store_token_parts(R, a.dr + ch * token_tiles(a.dv), a.dv, row0, w, lane);
    {
      // dX = dV = b dR; the operand of -e^G dX
      float y[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 be = *reinterpret_cast<const float2*>(gate + 128 + 8 * i);
        const float2 eg = *reinterpret_cast<const float2*>(gate + 8 * i);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          R[i][e] *= e & 1 ? be.y : be.x;
          y[i][e] = -(e & 1 ? eg.y : eg.x) * R[i][e];
        }
      }
      put_tiles<3>(own + W::kW, w, y[0], y[1], lane);
    }
    {
      uint32_t bk[4][DK / 64][4];
      load_rows<DK>(bk, sk, w, lane);
      const float last = reinterpret_cast<const float*>(st + W::kGate)[63];
      team_bar(slice);
      // dS = e^{G_63} dS' + (scale e^G dO)^T Q - (e^G dX)^T K, this warp's columns
      float acc[DK / 32][4];
      outer_rows<DK>(acc, own + W::kW, bk, lane);
#pragma unroll
      for (int j = 0; j < DK / 32; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[j][e] = last * S[j][e] + acc[j][e];
      load_rows<DK>(bk, sq, w, lane);
      outer_rows<DK>(acc, own + W::kY, bk, lane);
#pragma unroll
      for (int j = 0; j < DK / 32; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[j][e] += acc[j][e];
      // every warp is past this chunk's
      put_state<DK, true>(own, S, w, lane, snapshot(c - 1), row0, a.dv);
    }
    // this warp's operand of dU0 is no longer read: its place stages dV
    const int n = min(kDeltaChunk, len - c * kDeltaChunk) - 16 * w;
    const int64_t orow = b * a.T + tok0 + int64_t(c) * kDeltaChunk + 16 * w;
    store_tokens(R, own + W::kX + w * 3 * kOperand, a.dvp + (orow * a.Hv + h) * a.dv + row0, int64_t(a.Hv) * a.dv,
                 n, lane);
  }
  if (a.dstate_in) store_state<DK>(S, a.dstate_in, srow, w, lane);
}

// --------------------------------------------------------- dq, dk, dg, dbeta
struct KeyGradArgs {
  HeadView q, k, dout;
  GateView g;
  int Hk, Hv, dv, T;
  DeltaMap map;
  float scale;
  const unsigned char* blocks;
  const unsigned char *snap, *dsnap, *e, *dr;
  int64_t block_bytes, gate_at;  // a chunk's block, and the gates in it
  __nv_bfloat16 *dq, *dk;
  float *dg, *dbeta;
  unsigned int* status;
};

constexpr int kKeyThreads = 512;

// Shared memory, for a pass over a panel of kPanel rows of dv.  Every operand is tiles
// of 128-byte rows, swizzled:
//   dO      [64 tokens, then 64 rows of zeros][dv]
//   dR, E   [3 parts][rows of dv][64 tokens]
//   S, dS'  [3 parts][pieces of 8 dk][rows of dv], not swizzled
//   Q, K    [blocks of 64 dk][64 tokens of Q, then of K]
//   P       [3 parts][P1, L][64 rows][64 columns], over dR, which is used up by then
// and what dg is summed from.
struct KeyShape {
  static constexpr uint32_t kSeg = 8192;
  static constexpr uint32_t kZero = kSeg;  // the zeros below dO
  static constexpr uint32_t kX = 2 * kSeg, kTokPart = kSeg;
  static constexpr uint32_t kP = kX, kPPart = 2 * kSeg;
  static constexpr uint32_t kE = kP + 3 * kPPart;
  static constexpr uint32_t kState = kE + 3 * kTokPart, kStatePart = 2 * kSeg, kState1 = kState + 3 * kStatePart;
  static constexpr uint32_t kQ = kState1 + 3 * kStatePart, kBlock = 2 * kSeg, kK = kQ + kSeg;
  static constexpr uint32_t kSums = kQ + 2 * kBlock;
};
struct KeySums {
  Pair G[2][kDeltaChunk];         // of this head and the next
  float gate[2][3][kDeltaChunk];  // e^G, e^{G_63 - G}, beta
  float a[4][128];                // by quarter of dk: a_i, its part of dq and that of dk
  float c[4][kDeltaChunk];
  float b[4][128];                // sums of B_ij over a quarter of the columns
  float r[4][kDeltaChunk];        // by 32 rows i: sum of B_ij over i >= t > j
  float d[kKeyThreads / 32];      // <dS', S>
};
struct KeyBars {
  uint64_t s, r, e, d;  // S, dR, E, dS' are loaded
  uint64_t done_s, done_d, done_p;
  uint32_t tmem;
  int abort;
};
// Columns of tensor memory: [dO; dR] E^T; [dO; dR] S, then P1^T Q + L^T K; [0; E] dS';
// [P1; L] K; [Q; K] K^T.
constexpr uint32_t kTmP = 0, kTmS = 64, kTmD = 192, kTmK = 320, kTmQ = 448;

// dg of a chunk and head, by one warp, two tokens a lane.  Sums run from the far end
// (nothing is subtracted), so small ones keep their digits.
__device__ __forceinline__ void gate_gradient(const KeySums& s, int set, float* dg, int64_t stride, int n, int lane) {
  const int t0 = 2 * lane;
  float a[2], c[2], r[2], d = lane < kKeyThreads / 32 ? s.d[lane] : 0.f;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    a[i] = c[i] = r[i] = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      a[i] += s.a[w][t0 + i] + s.a[w][64 + t0 + i];
      c[i] += s.c[w][t0 + i];
      r[i] += s.r[w][t0 + i];
    }
  }
#pragma unroll
  for (int m = 16; m; m >>= 1) d += __shfl_xor_sync(~0u, d, m);
  d = s.gate[set][0][63] == 0.f ? 0.f : d * s.gate[set][0][63];
  float after = a[0] + a[1], before = c[0] + c[1];
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const float x = __shfl_down_sync(~0u, after, m), y = __shfl_up_sync(~0u, before, m);
    if (lane + m < 32) after += x;
    if (lane >= m) before += y;
  }
  after = __shfl_down_sync(~0u, after, 1);
  before = __shfl_up_sync(~0u, before, 1);
  if (lane == 31) after = 0.f;
  if (lane == 0) before = 0.f;
  if (t0 < n) dg[t0 * stride] = (after + a[1] + a[0]) + before + r[0] + d;
  if (t0 + 1 < n) dg[(t0 + 1) * stride] = (after + a[1]) + (before + c[0]) + r[1] + d;
}

// One (chunk, key head), on the tensor cores: 128 accumulator rows, dq's 64
// tokens above dk's 64.  Once: [Q; K] K^T.  For each value head that shares the key
// head, in order, with U = b E and dX = b dR, by panels of dv:
//   [dO; dR] E^T, added over the panels in registers -> with the decays and betas P1
//     (rows of dq) and L (below the diagonal); its lower diagonal is dbeta; with
//     [Q; K] K^T the B_ij of dg
//   [dO; dR] S, [0; E] dS': scaled by row and added in registers; dotted with q and k
//     the a_i and c_j of dg
// and then [P1; L] K and [0; P1^T] Q + [0; L^T] K, added in registers.
// A transposed left operand is a second group of 64 rows below one of zeros.
// Operands that are not bf16 as given have three parts, and products of parts p, r
// are kept for p + r < 3, as in the walks.  Sums over panels and heads are in
// registers because each addition in tensor memory rounds the full-size sum towards
// zero (in tensor memory dbeta's error in the Frobenius norm was 7.7e-7, now 3.1e-7).
// What a pass has used up is loaded anew at once, so that the next one's operands
// arrive under its remaining products and sums.  128 chunks of 10 key heads, two value
// heads of 128 x 128 each: 311 us, of which 112 would be the bytes (755 MB, mostly
// states) and 130 the products; products and the sums that wait for them take turns.
// (With the next head's operands prefetched into L2 as well some 40 us more: they are
// evicted again, and a quarter of the bytes is read twice.)
template <int DK>
__global__ void __launch_bounds__(kKeyThreads, 1) delta_key_grad_kernel(KeyGradArgs a) {
  extern __shared__ unsigned char smem_raw[];
  using W = KeyShape;
  constexpr int NB = DK / 64;  // blocks of dk
  constexpr int HC = DK / 4;   // columns a thread
  unsigned char* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);  // an offset: its loads stay shared ones
  const uint32_t sb = smem_u32(smem);
  KeySums& sums = *reinterpret_cast<KeySums*>(smem + W::kSums);
  KeyBars* bars = reinterpret_cast<KeyBars*>(smem + W::kSums + sizeof(KeySums));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row = (warp & 3) * 32 + lane, quarter = warp >> 2;  // accumulator row, quarter of the columns
  const int tok = row & 63;
  const bool is_k = row >= 64;
  if (tid == 0) {
    for (uint64_t* bar : {&bars->s, &bars->r, &bars->e, &bars->d, &bars->done_s, &bars->done_d, &bars->done_p})
      mbar_init(bar, 1);
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(&bars->tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tm = bars->tmem;
  const uint32_t trow = tm + (uint32_t((warp & 3) * 32) << 16);
  griddep_wait();
  griddep_launch_dependents();
  const int chunk = blockIdx.x, hk = blockIdx.y, group = a.Hv / a.Hk, h_end = (hk + 1) * group;
  const int s = a.map.doc_of(chunk);
  const int t0 = (chunk - a.map.chunk0(s)) * kDeltaChunk;
  const int n = min(kDeltaChunk, a.map.len(s) - t0);
  const int64_t b = a.map.row(s), t = a.map.start(s) + t0;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (!mbar_wait(bar, parity, &bars->abort)) raise_abort(&bars->abort, a.status, kStatusTimeout);
  };
  // Loads of a panel's operands, by one thread: three parts each.
  auto head = [&](int h) { return int64_t(chunk) * a.Hv + h; };
  auto load_states = [&](const unsigned char* from, int h, int v0, uint32_t to, uint64_t* bar) {
    if (aborted(&bars->abort)) return;
    const uint32_t bytes = uint32_t(min(kPanel, a.dv - v0)) * DK * 2;
    from += head(h) * state_parts(a.dv, DK) + state_parts(v0, DK);
    mbar_arrive_expect_tx(bar, 3 * bytes);
    for (int p = 0; p < 3; ++p) bulk_load(smem + to + p * W::kStatePart, from + p * bytes, bytes, bar);
  };
  auto load_tokens = [&](const unsigned char* from, int h, int v0, uint32_t to, uint64_t* bar) {
    if (aborted(&bars->abort)) return;
    const uint32_t bytes = uint32_t(min(kPanel, a.dv - v0)) * 128;
    from += head(h) * token_tiles(a.dv) + int64_t(v0) * 128;
    mbar_arrive_expect_tx(bar, 3 * bytes);
    for (int p = 0; p < 3; ++p) bulk_load(smem + to + p * W::kTokPart, from + int64_t(p) * a.dv * 128, bytes, bar);
  };
  // dO of a panel: one piece of 8 a thread
  static_assert(kKeyThreads == kDeltaChunk * 8, "a piece of dO, and of the zeros, a thread");
  auto load_do = [&](int h, int v0) {
    const int r = tid >> 3, p = tid & 7;
    if (p * 8 < min(kPanel, a.dv - v0)) {
      unsigned char* d = smem + tile_at<8>(r, p);
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.dout.data) + b * a.dout.sb + t * a.dout.st +
                                 h * a.dout.sh + v0 + p * 8 + (r < n ? r * a.dout.st : 0);
      if (a.dout.vec)
        cp16(smem_u32(d), src, r < n);
      else if (r < n)
        store_piece(d, src);
      else
        *reinterpret_cast<uint4*>(d) = make_uint4(0, 0, 0, 0);
    }
    cp_commit();
  };
  // a head's gates and their sums, by two warps
  auto load_gates = [&](int h) {
    const int set = h & 1;
    if (warp == 1) {
      const float* from = reinterpret_cast<const float*>(a.blocks + head(h) * a.block_bytes + a.gate_at);
#pragma unroll
      for (int i = 0; i < 3 * kDeltaChunk; i += 32) (&sums.gate[set][0][0])[i + lane] = from[i + lane];
    } else if (warp == 2) {
      gate_sums(a.g, b, t, h, n, lane, sums.G[set]);
    }
  };
  if (tid == 0) {
    load_tokens(a.dr, hk * group, 0, W::kX, &bars->r);
    load_tokens(a.e, hk * group, 0, W::kE, &bars->e);
    load_states(a.snap, hk * group, 0, W::kState, &bars->s);
    load_states(a.dsnap, hk * group, 0, W::kState1, &bars->d);
  }
  __syncwarp();
  {
    const auto* kp = static_cast<const __nv_bfloat16*>(a.k.data) + b * a.k.sb + t * a.k.st + hk * a.k.sh;
    const auto* qp = static_cast<const __nv_bfloat16*>(a.q.data) + b * a.q.sb + t * a.q.st + hk * a.q.sh;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      load_tile<8>(smem + W::kQ + i * W::kBlock, qp + 64 * i, a.q.st, n, a.q.vec, tid, kKeyThreads);
      load_tile<8>(smem + W::kK + i * W::kBlock, kp + 64 * i, a.k.st, n, a.k.vec, tid, kKeyThreads);
    }
    *reinterpret_cast<uint4*>(smem + W::kZero + tid * 16) = make_uint4(0, 0, 0, 0);
  }
  load_do(hk * group, 0);
  load_gates(hk * group);
  // left operand by rows or transposed; right operands have their rows along the
  // sum, but for K in [Q; K] K^T
  constexpr uint32_t id_p = idesc_bf16_f32(128, 64, false, true), id_pt = idesc_bf16_f32(128, 64, true, true);
  constexpr uint32_t id_s = idesc_bf16_f32(128, DK, false, true), id_st = idesc_bf16_f32(128, DK, true, true);
  constexpr uint32_t id_q = idesc_bf16_f32(128, 64, false, false);
  // low words of descriptors: an operand; one below 64 rows of zeros
  uint32_t base = __shfl_sync(~0u, sb, 0) >> 4;
  const uint32_t tmu = __shfl_sync(~0u, tm, 0);
  auto lo = [&](uint32_t at, uint32_t lbo = 16) { return base + ((at >> 4) | (lbo >> 4) << 16); };
  auto below = [&](uint32_t at) { return base + ((W::kZero >> 4) | ((at - W::kZero) >> 4) << 16); };
  float acc[HC], P[16];
#pragma unroll
  for (int e = 0; e < HC; ++e) acc[e] = 0.f;
  // this thread's row of [Q; K], 8 columns from `piece` of its quarter, dotted with v
  auto dot_row = [&](int piece, const float* v) {
    const int at = quarter * (HC / 8) + piece;
    const uint4 x = *reinterpret_cast<const uint4*>(smem + W::kQ + (at >> 3) * W::kBlock + tile_at<8>(row, at & 7));
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = unpack_bf16x2(w[e]);
      sum += f.x * v[2 * e] + f.y * v[2 * e + 1];
    }
    return sum;
  };
  uint32_t it = 0;  // passes over a panel
  for (int h = hk * group; h < h_end; ++h) {
    const int set = h & 1;
    float dot = 0.f, part_a = 0.f, part_c = 0.f;  // <dS', S>; this row's a_i and c_j
#pragma unroll
    for (int i = 0; i < 16; ++i) P[i] = 0.f;
    for (int v0 = 0; v0 < a.dv; v0 += kPanel, ++it) {
      const int width = min(kPanel, a.dv - v0), steps = width / 16;
      const uint32_t par = it & 1;
      const bool last = v0 + kPanel >= a.dv;
      const int next_h = last ? h + 1 : h, next_v = last ? 0 : v0 + kPanel;
      const bool more = next_h < h_end;
      // the states' descriptor: core matrices of 8 rows of dv by 16 bytes of dk,
      // 128 bytes apart along the rows, width * 16 along dk
      const uint32_t state_hi = uint32_t(width) | (1u << 14);
      cp_wait<0>();
      fence_proxy_async_smem();
      tc_fence_before_sync();
      __syncthreads();  // dO; the accumulators are read, last pass's sums too
      if (warp == 0) {
        const uint32_t on = elect_one();
        asm volatile("" : "+r"(base));  // descriptors are worked out anew, not kept in registers
        tc_fence_after_sync();
        if (it == 0)
#pragma unroll
          for (int ks = 0; ks < DK / 16; ++ks)
            mma_ss(on, tmu + kTmQ, lo(W::kQ + (ks >> 2) * W::kBlock + (ks & 3) * 32),
                   lo(W::kK + (ks >> 2) * W::kBlock + (ks & 3) * 32), id_q, ks > 0);
        wait(&bars->r, par);
        wait(&bars->e, par);
        wait(&bars->s, par);
        // small terms first; dO is exact, so it has no other parts (unrolled: with
        // descriptors worked out in loops, each product cost its issuer 100 cycles)
#pragma unroll
        for (int sum = 2; sum >= 0; --sum)
#pragma unroll
          for (int p = 0; p <= sum; ++p)
#pragma unroll
            for (int ks = 0; ks < kPanel / 16; ++ks)
              if (ks < steps) {
                const uint32_t dos = lo(ks * 32), be = lo(W::kE + (sum - p) * W::kTokPart + ks * 2048);
                const uint32_t bs = lo(W::kState + (sum - p) * W::kStatePart + ks * 256, 128);
                const uint32_t ax = below(W::kX + p * W::kTokPart + ks * 2048);
                if (p == 0) {
                  mma_ss(on, tmu + kTmP, dos, be, id_p, sum < 2 || ks > 0);
                  mma_ss(on, tmu + kTmS, dos, bs, id_s, sum < 2 || ks > 0, state_hi);
                }
                mma_ss(on, tmu + kTmP, ax, be, id_pt, 1);
                mma_ss(on, tmu + kTmS, ax, bs, id_st, 1, state_hi);
              }
        commit(on, &bars->done_s);
        wait(&bars->d, par);
#pragma unroll
        for (int sum = 2; sum >= 0; --sum)
#pragma unroll
          for (int p = 0; p <= sum; ++p)
#pragma unroll
            for (int ks = 0; ks < kPanel / 16; ++ks)
              if (ks < steps)
                mma_ss(on, tmu + kTmD, below(W::kE + p * W::kTokPart + ks * 2048),
                       lo(W::kState1 + (sum - p) * W::kStatePart + ks * 256, 128), id_st, sum < 2 || p > 0 || ks > 0,
                       state_hi);
        commit(on, &bars->done_d);
      }
      __syncwarp();
      // <dS', S>, shared by the other warps
      wait(&bars->s, par);
      wait(&bars->d, par);
      for (int i = warp ? tid - 32 : width * (DK / 8); i < width * (DK / 8); i += kKeyThreads - 32) {
        float x[2][8];
#pragma unroll
        for (int which = 0; which < 2; ++which) {
          const unsigned char* at = smem + (which ? W::kState1 : W::kState) + i * 16;
          uint32_t w[3][4];
#pragma unroll
          for (int p = 0; p < 3; ++p) {
            const uint4 u = *reinterpret_cast<const uint4*>(at + p * W::kStatePart);
            w[p][0] = u.x;
            w[p][1] = u.y;
            w[p][2] = u.z;
            w[p][3] = u.w;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 hi = unpack_bf16x2(w[0][e]), mid = unpack_bf16x2(w[1][e]), low = unpack_bf16x2(w[2][e]);
            x[which][2 * e] = hi.x + (mid.x + low.x);
            x[which][2 * e + 1] = hi.y + (mid.y + low.y);
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) dot += x[0][e] * x[1][e];
      }
      const float eg = sums.gate[set][0][tok], bt = sums.gate[set][2][tok];
      wait(&bars->done_s, par);
      tc_fence_after_sync();
      {
        float v[16];
        read16(trow + kTmP + 16 * quarter, v);
#pragma unroll
        for (int i = 0; i < 16; ++i) P[i] += v[i];
        const float m = is_k ? -eg * bt : a.scale * eg;
#pragma unroll
        for (int c0 = 0; c0 < HC; c0 += 16) {
          read16(trow + kTmS + quarter * HC + c0, v);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            v[e] = eg == 0.f ? 0.f : v[e] * m;  // (a state before a reset may be anything)
            acc[c0 + e] += v[e];
          }
          part_a += dot_row(c0 / 8, v) + dot_row(c0 / 8 + 1, v + 8);
        }
      }
      tc_fence_before_sync();
      __syncthreads();  // S, dR and dO are used up
      if (more) {
        if (tid == 0) {
          load_states(a.snap, next_h, next_v, W::kState, &bars->s);
          if (!last) load_tokens(a.dr, next_h, next_v, W::kX, &bars->r);
        }
        __syncwarp();
        load_do(next_h, next_v);
        if (last) load_gates(next_h);
      }
      if (last) {
        // P1 and L: this thread's row, 16 columns
        float B[16], sum = 0.f;
        read16(trow + kTmQ + 16 * quarter, B);
        const Pair g = sums.G[set][tok];
#pragma unroll
        for (int piece = 0; piece < 2; ++piece) {
          uint32_t p[4][3];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float x[2];
#pragma unroll
            for (int f = 0; f < 2; ++f) {
              const int i = piece * 8 + 2 * e + f, c = 16 * quarter + i;
              if (is_k && c == tok && tok < n) a.dbeta[(b * a.T + t + tok) * a.Hv + h] = P[i];  // dR.E
              const bool on = is_k ? c < tok : c <= tok;
              const float d = on ? decay(g, sums.G[set][c]) * sums.gate[set][2][c] : 0.f;
              x[f] = on ? (is_k ? -bt * d : a.scale * d) * P[i] : 0.f;
              B[i] = c < tok ? x[f] * B[i] : 0.f;
              sum += B[i];
            }
            split2<3>(x[0], x[1], p[e]);
          }
          unsigned char* to = smem + W::kP + (is_k ? W::kSeg : 0) + tile_at<8>(tok, 2 * quarter + piece);
#pragma unroll
          for (int q = 0; q < 3; ++q)
            *reinterpret_cast<uint4*>(to + q * W::kPPart) = make_uint4(p[0][q], p[1][q], p[2][q], p[3][q]);
        }
        sums.b[quarter][row] = sum;
        fence_proxy_async_smem();
        tc_fence_before_sync();
        __syncthreads();
        if (warp == 0) {
          const uint32_t on = elect_one();
          asm volatile("" : "+r"(base));
          tc_fence_after_sync();
#pragma unroll
          for (int p = 2; p >= 0; --p)
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
              const uint32_t pt = W::kP + p * W::kPPart + ks * 2048;
              const uint32_t bk = lo(W::kK + ks * 2048, W::kBlock), bq = lo(W::kQ + ks * 2048, W::kBlock);
              mma_ss(on, tmu + kTmK, lo(W::kP + p * W::kPPart + ks * 32), bk, id_s, p < 2 || ks > 0);
              mma_ss(on, tmu + kTmS, below(pt), bq, id_st, p < 2 || ks > 0);
              mma_ss(on, tmu + kTmS, below(pt + W::kSeg), bk, id_st, 1);
            }
          commit(on, &bars->done_p);
        }
        __syncwarp();
        // sum of B_ij over this warp's rows i >= t and the columns j < t
        float before = 0.f;
        for (int w = 0; w < quarter; ++w) before += sums.b[w][row];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float x = B[i];
          B[i] = 16 * quarter + i <= tok ? before : 0.f;
          before += x;
        }
        store_row_sums(B, sums.r[warp & 3] + 16 * quarter, lane);
      }
      wait(&bars->done_d, par);
      tc_fence_after_sync();
      if (more && tid == 0) {
        load_tokens(a.e, next_h, next_v, W::kE, &bars->e);
        load_states(a.dsnap, next_h, next_v, W::kState1, &bars->d);
      }
      __syncwarp();
      if (is_k) {
        const float m = sums.gate[set][1][tok] * bt;
#pragma unroll
        for (int c0 = 0; c0 < HC; c0 += 16) {
          float v[16];
          read16(trow + kTmD + quarter * HC + c0, v);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            v[e] *= m;
            acc[c0 + e] += v[e];
          }
          part_c += dot_row(c0 / 8, v) + dot_row(c0 / 8 + 1, v + 8);
        }
      }
      if (last) {
        sums.a[quarter][row] = part_a;
        if (is_k) sums.c[quarter][tok] = part_c;
#pragma unroll
        for (int m = 16; m; m >>= 1) dot += __shfl_xor_sync(~0u, dot, m);
        if (lane == 0) sums.d[warp] = dot;
        wait(&bars->done_p, (h - hk * group) & 1);
        tc_fence_after_sync();
        if (more && tid == 0) load_tokens(a.dr, next_h, next_v, W::kX, &bars->r);
        __syncwarp();
#pragma unroll
        for (int c0 = 0; c0 < HC; c0 += 16) {
          float v[16];
          read16(trow + kTmK + quarter * HC + c0, v);
#pragma unroll
          for (int e = 0; e < 16; ++e) acc[c0 + e] += v[e];
          if (is_k) {
            read16(trow + kTmS + quarter * HC + c0, v);
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[c0 + e] += v[e];
          }
        }
        tc_fence_before_sync();
        __syncthreads();
        // its sums are next written behind a barrier that this warp joins later
        if (warp == 3) gate_gradient(sums, set, a.dg + (b * a.T + t) * a.Hv + h, a.Hv, n, lane);
      }
    }
  }
  if (tok < n) {
    __nv_bfloat16* to = (is_k ? a.dk : a.dq) + ((b * a.T + t + tok) * a.Hk + hk) * DK + quarter * HC;
#pragma unroll
    for (int e = 0; e < HC; e += 8) {
      uint32_t w[4];
#pragma unroll
      for (int f = 0; f < 4; ++f) w[f] = pack_bf16x2(acc[e + 2 * f], acc[e + 2 * f + 1]);
      *reinterpret_cast<uint4*>(to + e) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  settle(&bars->abort);
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after_sync();
    tmem_dealloc(tm, 512);
  }
}

template <int DK>
cudaError_t run_team_reverse(const LaunchEnv& env, const ReverseArgs& r) {
  using W = ReverseShape<DK>;
  const int ns = walk_slices(r.map.ndocs, r.Hv, r.dv, env.num_sms);
  const cudaError_t e = cudaFuncSetAttribute(delta_reverse_kernel<DK>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, W::smem(2));
  if (e != cudaSuccess) return e;
  return launch_pdl(delta_reverse_kernel<DK>, dim3(unsigned(r.map.ndocs * r.Hv * (r.dv / (16 * ns)))),
                    dim3(kTeam * ns + 32), W::smem(ns), env.stream, r);
}

template <int DK>
cudaError_t run_key_grad(const LaunchEnv& env, const KeyGradArgs& g) {
  constexpr int smem = KeyShape::kSums + int(sizeof(KeySums) + sizeof(KeyBars)) + 1024;
  const cudaError_t e = cudaFuncSetAttribute(delta_key_grad_kernel<DK>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(delta_key_grad_kernel<DK>, dim3(unsigned(g.map.nchunks), unsigned(g.Hk)),
                    dim3(kKeyThreads), smem, env.stream, g);
}

// Scratch after the blocks, in bytes.
struct GradLayout {
  size_t snap, dsnap, e, dr, total;
};
GradLayout grad_layout(int64_t nchunks, int Hv, int dk, int dv) {
  auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  const size_t heads = size_t(nchunks) * size_t(Hv);
  GradLayout L;
  size_t at = up(heads * kWideGrad);  // the larger of the blocks' two forms
  auto take = [&](size_t* where, size_t bytes) {
    *where = at;
    at += up(bytes);
  };
  take(&L.snap, heads * size_t(state_parts(dv, dk)));
  take(&L.dsnap, heads * size_t(state_parts(dv, dk)));
  take(&L.e, heads * size_t(token_tiles(dv)));
  take(&L.dr, heads * size_t(token_tiles(dv)));
  L.total = at;
  return L;
}

}  // namespace

size_t delta_grad_scratch(int64_t nchunks, int Hv, int dk, int dv) { return grad_layout(nchunks, Hv, dk, dv).total; }

cudaError_t launch_delta_grad(const LaunchEnv& env, const DeltaGradArgs& a) {
  const DeltaArgs& f = a.f;
  const GradLayout L = grad_layout(f.map.nchunks, f.Hv, f.dk, f.dv);
  cudaError_t e = cudaSuccess;
  const bool by_head = delta_by_head(f.map.ndocs, f.Hv, f.dv, env.num_sms);
  if (f.map.nchunks > 0 && (e = launch_delta_prepare(env, f, f.ws, true, by_head)) != cudaSuccess) return e;
  DeltaSave save;
  save.snap = f.ws + L.snap;
  save.e = f.ws + L.e;
  e = by_head ? launch_head_walk(env, f, f.ws, &save) : launch_team_walk(env, f, f.ws, &save);
  if (e != cudaSuccess) return e;
  ReverseArgs r;
  r.q = f.q;
  r.k = f.k;
  r.dout = a.dout;
  r.Hk = f.Hk;
  r.Hv = f.Hv;
  r.dv = f.dv;
  r.T = f.T;
  r.map = f.map;
  r.scale = f.scale;
  r.blocks = f.ws;
  r.status = env.status;
  r.dstate_out = a.dstate_out;
  r.dstate_in = a.dstate_in;
  r.dvp = static_cast<__nv_bfloat16*>(a.dv);
  r.dr = f.ws + L.dr;
  r.dsnap = f.ws + L.dsnap;
  KeyGradArgs g;
  g.q = f.q;
  g.k = f.k;
  g.dout = a.dout;
  g.g = f.g;
  g.Hk = f.Hk;
  g.Hv = f.Hv;
  g.dv = f.dv;
  g.T = f.T;
  g.map = f.map;
  g.scale = f.scale;
  g.blocks = f.ws;
  g.snap = save.snap;
  g.dsnap = r.dsnap;
  g.e = save.e;
  g.dr = r.dr;
  g.status = env.status;
  g.dq = static_cast<__nv_bfloat16*>(a.dq);
  g.dk = static_cast<__nv_bfloat16*>(a.dk);
  g.dg = a.dg;
  g.dbeta = a.dbeta;
  g.block_bytes = by_head ? kWideGrad : kBlkGrad;
  g.gate_at = by_head ? kWideGate : kBlkGate;
  if (by_head)
    e = launch_head_reverse(env, r, f.dk);
  else
    e = f.dk == 64 ? run_team_reverse<64>(env, r) : run_team_reverse<128>(env, r);
  if (e != cudaSuccess || f.map.nchunks == 0) return e;
  return f.dk == 64 ? run_key_grad<64>(env, g) : run_key_grad<128>(env, g);
}

}  // namespace ittt
