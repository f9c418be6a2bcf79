// k_delta.cu -- the gated delta rule, chunked and token by token.
//
//   S_t = a_t S_{t-1} + b_t (v_t - a_t S_{t-1} k_t) k_t^T,  a_t = e^{g_t},
//   o_t = scale S_t q_t                                     S: [dv x dk], fp32
//
// Over a chunk of 64 tokens that starts from S, with G the running sum of g:
//   X = V - e^G (K S^T)             what the tokens do not find in S
//   E = (I + B diag(b))^-1 X        B_ij = e^{G_i - G_j} k_i.k_j for j < i
//   O = scale e^G (Q S^T) + M (b E)     M_ij = scale e^{G_i - G_j} q_i.k_j, j <= i
//   S <- e^{G_63} S + (b E)^T (e^{G_63 - G} K)
// The inverse and M depend on q, k, g and b alone: a first kernel forms them
// for all chunks at once.  The second walks the chunks in order.
//
// 8192 tokens, 20 heads of 128 x 128 (10 key heads): 48 + 443 us.  The call's bytes
// would pass in 19 us and its products in 10; it is bound by the chain of 128
// chunks, 3.5 us each, of three products that wait for one another (token by token
// it would be 8192 steps of 0.9 us).  The output's products have 24-bit operands too,
// so that a bf16 output is the exact one's rounding; with 16 bits, which moved 0.3% of
// the outputs to the other neighbour, the walk took 398 us (heads of 64 x 64: 4096
// tokens of 16 heads 183 us then, 147 now, with the scores read where they are used).
#include <algorithm>

#include "delta.cuh"

namespace ittt {
namespace {

constexpr int kPrepThreads = 256;

struct PrepArgs {
  HeadView q, k;
  GateView g, beta;
  int Hk, Hv;
  DeltaMap map;
  float scale;
  unsigned char* blocks;
  bool wide;
};

// The part of the inverse T of I + C (C strictly lower triangular, 64 x 64)
// below its diagonal blocks, columns [16j, 16j + 16), by one warp:
//   T_ij = -T_ii sum_{j <= m < i} C_im T_mj,   i = j + 1 .. 3,
// transposed, so that each product's accumulators are the next one's left
// operand.  `c` holds C's blocks and `t` T's, three parts each, T_ii given.
__device__ __forceinline__ void solve_columns(unsigned char* t, uint32_t c, int j, int lane) {
  uint32_t ta[3][3][4];  // T_mj^T, m = j ..
  const uint32_t ts = smem_u32(t);
#pragma unroll
  for (int p = 0; p < 3; ++p) ldsm4_t(ta[0][p], ts + p * kImage + image_block(j, j) + block_km(lane));
#pragma unroll
  for (int d = 1; d < 4; ++d) {
    const int i = j + d;
    if (i > 3) break;
    float H[2][4], L[2][4], M[2][4];
    auto product = [&](const uint32_t (&xa)[3][4], uint32_t blk) {
      uint32_t b[3][4];
#pragma unroll
      for (int r = 0; r < 3; ++r) ldsm4(b[r], blk + r * kImage + block_nk(lane));
      mma2(L[0], L[1], xa[0], b[2]);
      mma2(M[0], M[1], xa[2], b[0]);
      mma2(L[0], L[1], xa[1], b[1]);
      mma2(M[0], M[1], xa[1], b[0]);
      mma2(L[0], L[1], xa[0], b[1]);
      mma2(H[0], H[1], xa[0], b[0]);
    };
    auto total = [&](float sign) {
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) H[n][e] = sign * (H[n][e] + (L[n][e] + M[n][e]));
    };
    zero(H);
    zero(L);
    zero(M);
#pragma unroll
    for (int m = 0; m < d; ++m) product(ta[m], c + image_block(i, j + m));
    total(-1.f);
    uint32_t xa[3][4];
    split_frag<3>(H[0], H[1], xa);
    zero(H);
    zero(L);
    zero(M);
    product(xa, ts + image_block(i, i));
    total(1.f);
    split_frag<3>(H[0], H[1], xa);
#pragma unroll
    for (int p = 0; p < 3; ++p) {
      // the left operand holds [column of j][token of i] pairs along i
      stsm4_t(ts + p * kImage + image_block(i, j) + block_at(8 * (lane >> 4) + (lane & 7), (lane >> 3) & 1),
              xa[p][0], xa[p][1], xa[p][2], xa[p][3]);
      if (d < 3)
#pragma unroll
        for (int e = 0; e < 4; ++e) ta[d < 3 ? d : 0][p][e] = xa[p][e];
    }
  }
}

// Shared memory: K and Q, over which the results are laid once the products are
// formed; C (its blocks below the diagonal ones, three parts) and its diagonal
// blocks in fp32, for one or two maps; running sums and betas.
template <int DK, bool GRAD>
struct PrepShape {
  static constexpr int kMaps = GRAD ? 2 : 1;
  static constexpr int kTile = kDeltaChunk * DK * 2;
  static constexpr int kOut = GRAD ? kBlkGrad : kBlkFwd;
  static constexpr int kC = 2 * kTile > kOut ? 2 * kTile : kOut;
  static constexpr int kDiag = kC + kMaps * 3 * kImage;
  static constexpr int kSums = kDiag + kMaps * 4 * 16 * 17 * 4;
  static constexpr int kSmem = kSums + kDeltaChunk * 12;
};

// One (chunk, head).  Eight warps form the lower blocks of K K^T and Q K^T (16
// rows and at most two blocks each) on the tensor cores.  The triangular inverse
// goes by 16 x 16 blocks: substitution for the four on the diagonal, one thread a
// column, then products for the others, one warp a column of blocks.  Every phase
// is short and waits for the one before, so what counts are warps an SM: with four
// a CTA the products' masks alone took 6700 of 22700 cycles, most of it one warp's.
// 6016 chunks and heads of dk 64: 115 us (125 with four warps), of which 26 would
// be its reads and writes.
template <int DK, bool GRAD>
__global__ void __launch_bounds__(kPrepThreads, GRAD ? 2 : 4) delta_prepare_kernel(PrepArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  using W = PrepShape<DK, GRAD>;
  constexpr int CH = DK / 8;
  unsigned char* tk = smem;
  unsigned char* tq = smem + W::kTile;
  float* diag = reinterpret_cast<float*>(smem + W::kDiag);  // [maps][4][16][17]
  Pair* G = reinterpret_cast<Pair*>(smem + W::kSums);
  float* beta = reinterpret_cast<float*>(G + kDeltaChunk);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int chunk = blockIdx.x, h = blockIdx.y, hk = h / (a.Hv / a.Hk);
  griddep_wait();
  griddep_launch_dependents();
  const int s = a.map.doc_of(chunk);
  const int t0 = (chunk - a.map.chunk0(s)) * kDeltaChunk;
  const int n = min(kDeltaChunk, a.map.len(s) - t0);
  const int64_t b = a.map.row(s), t = a.map.start(s) + t0;
  load_tile<CH>(tk, static_cast<const __nv_bfloat16*>(a.k.data) + b * a.k.sb + t * a.k.st + hk * a.k.sh,
                a.k.st, n, a.k.vec, tid, kPrepThreads);
  load_tile<CH>(tq, static_cast<const __nv_bfloat16*>(a.q.data) + b * a.q.sb + t * a.q.st + hk * a.q.sh,
                a.q.st, n, a.q.vec, tid, kPrepThreads);
  cp_commit();
  cp_wait<0>();
  __syncthreads();
  // rows [16 mine, 16 mine + 16) of the products, every other block of columns
  const int mine = warp & 3, other = warp >> 2;
  float kk[2][2][4], qk[2][2][4];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    zero(kk[x]);
    zero(qk[x]);
  }
  if (warp == 4) {  // the one warp without a block
    gate_sums(a.g, b, t, h, n, lane, G);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = 2 * lane + i;
      beta[r] = r < n ? a.beta.data[b * a.beta.sb + (t + r) * a.beta.st + h * a.beta.sh] : 0.f;
    }
  } else {
#pragma unroll
    for (int st = 0; st < DK / 16; ++st) {
      uint32_t ak[4], aq[4], bk[4];
      ldsm4(ak, smem_u32(tk) + addr_mk<CH>(mine, st, lane));
      ldsm4(aq, smem_u32(tq) + addr_mk<CH>(mine, st, lane));
#pragma unroll
      for (int x = 0; x < 2; ++x)
        if (other + 2 * x <= mine) {
          ldsm4(bk, smem_u32(tk) + addr_nk<CH>(2 * (other + 2 * x), st, lane));
          mma2(kk[x][0], kk[x][1], ak, bk);
          mma2(qk[x][0], qk[x][1], aq, bk);
        }
    }
  }
  __syncthreads();  // K and Q are no longer needed
  unsigned char* out = smem;  // laid out as the block
  float* gate = reinterpret_cast<float*>(out + kBlkGate);
  if (tid < kDeltaChunk) {
    gate[tid] = expf(G[tid].hi + G[tid].lo);
    gate[64 + tid] = decay(G[63], G[tid]);
    gate[128 + tid] = beta[tid];
  }
#pragma unroll
  for (int y = 0; y < 4; ++y)
    if (other + 2 * (y >> 1) <= mine)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int j = 2 * other + 4 * (y >> 1) + (y & 1);  // 8 columns
        const int r = 8 * half + (lane >> 2), i = 16 * mine + r, c = 8 * j + 2 * (lane & 3);
        const int at = image_block(mine, j >> 1) + block_at(r, j & 1) + 4 * (lane & 3);
        float x[2], m[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float d = c + e <= i ? decay(G[i], G[c + e]) : 0.f;
          m[e] = a.scale * d * qk[y >> 1][y & 1][2 * half + e];
          x[e] = c + e < i ? d * kk[y >> 1][y & 1][2 * half + e] : 0.f;
        }
        uint32_t p[3];
        split2<3>(m[0], m[1], p);
#pragma unroll
        for (int q = 0; q < 3; ++q) *reinterpret_cast<uint32_t*>(out + kBlkM + q * kImage + at) = p[q];
#pragma unroll
        for (int map = 0; map < W::kMaps; ++map) {
          // E map: B diag(beta); R map: diag(beta) B
          const float x0 = x[0] * (map ? beta[i] : beta[c]), x1 = x[1] * (map ? beta[i] : beta[c + 1]);
          if (j >= 2 * mine) {
            float* to = diag + ((map * 4 + mine) * 16 + r) * 17 + (c & 15);
            to[0] = x0;
            to[1] = x1;
          } else {
            split2<3>(x0, x1, p);
#pragma unroll
            for (int q = 0; q < 3; ++q)
              *reinterpret_cast<uint32_t*>(smem + W::kC + (map * 3 + q) * kImage + at) = p[q];
          }
        }
      }
  __syncthreads();
  if (tid < W::kMaps * 64) {
    // column `col` of diagonal block `blk`: (I + C) y = unit vector
    const int map = tid >> 6, blk = (tid >> 4) & 3, col = tid & 15;
    const float* cb = diag + (map * 4 + blk) * 16 * 17;
    unsigned char* img = out + (map ? kBlkR : kBlkE) + image_block(blk, blk) + 2 * (col & 7);
    float y[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s0 = 0.f, s1 = 0.f;
#pragma unroll
      for (int m = 0; m < i; ++m) (m & 1 ? s1 : s0) += cb[i * 17 + m] * y[m];
      y[i] = (i == col ? 1.f : 0.f) - (s0 + s1);
      float rest = y[i];
      unsigned char* at = img + block_at(i, col >> 3);
#pragma unroll
      for (int q = 0; q < 3; ++q) {
        const __nv_bfloat16 p = __float2bfloat16_rn(rest);
        *reinterpret_cast<__nv_bfloat16*>(at + q * kImage) = p;
        rest -= __bfloat162float(p);
      }
    }
  }
  __syncthreads();
  const uint32_t cs = smem_u32(smem + W::kC);
  if (mine < 3 && other < W::kMaps) solve_columns(out + (other ? kBlkR : kBlkE), cs + other * 3 * kImage, mine, lane);
  __syncthreads();
  if (!a.wide) {
    unsigned char* blk = a.blocks + (int64_t(chunk) * a.Hv + h) * W::kOut;
    for (int i = tid; i < W::kOut / 16; i += kPrepThreads)
      reinterpret_cast<uint4*>(blk)[i] = reinterpret_cast<const uint4*>(out)[i];
    return;
  }
  unsigned char* blk = a.blocks + (int64_t(chunk) * a.Hv + h) * (GRAD ? kWideGrad : kWideFwd);
  for (int x = tid; x < (GRAD ? 9 : 6) * 64 * 8; x += kPrepThreads) {
    const int part = x >> 9, i = (x >> 3) & 63, piece = x & 7;
    if (piece >> 1 > i >> 4) continue;
    const int from = part < 6 ? part * kImage : kBlkR + (part - 6) * kImage;
    const int to = part < 6 ? part * kWideTile : kWideR + (part - 6) * kWideTile;
    *reinterpret_cast<uint4*>(blk + to + tile_at<8>(i, piece)) = *reinterpret_cast<const uint4*>(
        out + from + image_block(i >> 4, piece >> 1) + block_at(i & 15, piece & 1));
  }
  if (tid < 48)
    reinterpret_cast<uint4*>(blk + kWideGate)[tid] = reinterpret_cast<const uint4*>(out + kBlkGate)[tid];
}

template <int DK, bool GRAD>
cudaError_t run_prepare(const LaunchEnv& env, const PrepArgs& p) {
  constexpr int smem = PrepShape<DK, GRAD>::kSmem;
  const cudaError_t e = cudaFuncSetAttribute(delta_prepare_kernel<DK, GRAD>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(delta_prepare_kernel<DK, GRAD>, dim3(unsigned(p.map.nchunks), unsigned(p.Hv)),
                    dim3(kPrepThreads), smem, env.stream, p);
}

// --------------------------------------------------------------------- walk
struct WalkArgs {
  HeadView q, k, v;
  int Hk, Hv, dv, T;
  DeltaMap map;
  float scale;
  const float* state_in;
  float* state_out;
  void* out;
  bool out_fp32;
  const unsigned char* blocks;
  unsigned int* status;
  DeltaSave save;  // SAVE only
};

// Shared memory of a CTA of `ns` slices: two stages (K, E map, gates, V, and for the
// output Q and the scores), then what each slice's warps exchange.
template <int DK, bool SAVE>
struct WalkShape {
  static constexpr int kTile = kDeltaChunk * DK * 2;
  static constexpr int kMap = (SAVE ? 1 : 2) * kTile;
  static constexpr int kMaps = (SAVE ? 3 : 6) * kImage;
  static constexpr int kGate = kMap + kMaps;
  static constexpr int kCols = kGate + 1024;
  static constexpr int kX = DK / 16 * 3 * kOperand;  // operands of X, after the state's
  static constexpr int kW = kX + 12 * kOperand;      // of e^{G_63 - G} U
  static constexpr int kU = kW + 12 * kOperand;      // of U
  static constexpr int kOwn = kU + (SAVE ? 0 : 12 * kOperand);
  static __host__ __device__ constexpr int stage(int ns) {
    return kCols + kDeltaChunk * (2 * ns + 1) * 16;
  }
  static __host__ __device__ constexpr int smem(int ns) {
    return 2 * stage(ns) + ns * kOwn + int(sizeof(StageBars));
  }
};

// One (sequence, head) and `ns` = blockDim.x / 128 slices of its dv rows, a team
// of four warps each, and a warp that loads.  SAVE: the gradient's forward pass, which
// writes no output and keeps the states at the chunks' starts and E.
template <int DK, bool SAVE>
__global__ void __launch_bounds__(2 * kTeam + 32) delta_walk_kernel(WalkArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  using W = WalkShape<DK, SAVE>;
  const int ns = blockDim.x / kTeam, tid = threadIdx.x, lane = tid & 31, slice = tid / kTeam;
  // the teams take their tokens in opposite orders: the triangle's long rows of
  // one share a scheduler with the short rows of the other
  const int w = slice & 1 ? 3 - ((tid >> 5) & 3) : (tid >> 5) & 3;
  const int pieces = 2 * ns, pitch = (pieces + 1) * 16;
  const int stage_bytes = W::stage(ns);
  const int parts = a.dv / (16 * ns);
  const int h = (blockIdx.x / parts) % a.Hv, s = blockIdx.x / (parts * a.Hv);
  const int col0 = (blockIdx.x % parts) * 16 * ns, row0 = col0 + 16 * slice;
  const int g4 = lane >> 2, t2 = 2 * (lane & 3);
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
    const auto* vp = static_cast<const __nv_bfloat16*>(a.v.data) + b * a.v.sb + tok0 * a.v.st + h * a.v.sh + col0;
    for (int c = 0; c <= nchunks; ++c) {
      if (c < nchunks) {
        unsigned char* st = smem + (c & 1) * stage_bytes;
        const int n = min(kDeltaChunk, len - c * kDeltaChunk);
        const int64_t t = int64_t(c) * kDeltaChunk;
        if (lane == 0) {
          const unsigned char* blk = a.blocks + ((chunk0 + c) * a.Hv + h) * int64_t(SAVE ? kBlkGrad : kBlkFwd);
          mbar_arrive_expect_tx(&bars->full[c & 1], W::kMaps + 768);
          bulk_load(st + W::kMap, blk, W::kMaps, &bars->full[c & 1]);
          bulk_load(st + W::kGate, blk + kBlkGate, 768, &bars->full[c & 1]);
        }
        warp_load_tile<DK / 8>(st, kp + t * a.k.st, a.k.st, n, a.k.vec, lane);
        if constexpr (!SAVE) warp_load_tile<DK / 8>(st + W::kTile, qp + t * a.q.st, a.q.st, n, a.q.vec, lane);
        load_cols(st + W::kCols, vp + t * a.v.st, a.v.st, pieces, n, a.v.vec, lane, 32);
        cp_wait_all();
      }
      // chunk c is in its stage; the teams are done with chunk c - 1
      if (__syncthreads_or(0)) break;
    }
    settle(&bars->abort);
    return;
  }

  float S[DK / 32][4];
  const int64_t srow = (int64_t(s) * a.Hv + h) * a.dv + row0;
  load_state<DK>(S, a.state_in, srow, w, lane);
  auto snapshot = [&](int c) {
    return SAVE && c < nchunks ? a.save.snap + ((chunk0 + c) * a.Hv + h) * state_parts(a.dv, DK) : nullptr;
  };
  put_state<DK, SAVE>(own, S, w, lane, snapshot(0), row0, a.dv);
  bool late = false;
  for (int c = 0;; ++c) {
    if (__syncthreads_or(late) || c == nchunks) break;
    late = wait_block(bars, c, a.status);
    const unsigned char* st = smem + (c & 1) * stage_bytes;
    const uint32_t sk = smem_u32(st), se = sk + W::kMap;
    const float* gate = reinterpret_cast<const float*>(st + W::kGate) + 16 * w + t2;  // this warp's tokens
    const int64_t ch = (chunk0 + c) * a.Hv + h;
    float X[2][4], O[2][4];
    state_times_rows<DK, SAVE ? 0 : 3>(own, sk, sk + W::kTile, w, lane, X, O);
    {
      // X = V - e^G (K S^T), O = scale e^G (Q S^T)
      uint32_t v[4];
      load_cols_t(v, sk + W::kCols + 32 * slice, pitch, w, lane);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 eg = *reinterpret_cast<const float2*>(gate + 8 * i);
        const float2 v0 = unpack_bf16x2(v[2 * i]), v1 = unpack_bf16x2(v[2 * i + 1]);
        // a decay of zero clears a state that is not finite too
        X[i][0] = eg.x == 0.f ? v0.x : v0.x - eg.x * X[i][0];
        X[i][1] = eg.y == 0.f ? v0.y : v0.y - eg.y * X[i][1];
        X[i][2] = eg.x == 0.f ? v1.x : v1.x - eg.x * X[i][2];
        X[i][3] = eg.y == 0.f ? v1.y : v1.y - eg.y * X[i][3];
        if constexpr (!SAVE) {
          O[i][0] = eg.x == 0.f ? 0.f : a.scale * eg.x * O[i][0];
          O[i][1] = eg.y == 0.f ? 0.f : a.scale * eg.y * O[i][1];
          O[i][2] = eg.x == 0.f ? 0.f : a.scale * eg.x * O[i][2];
          O[i][3] = eg.y == 0.f ? 0.f : a.scale * eg.y * O[i][3];
        }
      }
      put_tiles<3>(own + W::kX, w, X[0], X[1], lane);
    }
    float U[2][4];
    {
      uint32_t be[4][3][4];
      load_map<false, 3>(be, se, w, lane);
      team_bar(slice);
      map_tokens<false, 3>(own + W::kX, be, w, lane, U);  // E
    }
    if constexpr (SAVE) store_token_parts(U, a.save.e + ch * token_tiles(a.dv), a.dv, row0, w, lane);
    {
      // U = b E and e^{G_63 - G} U
      float V[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 be = *reinterpret_cast<const float2*>(gate + 128 + 8 * i);
        const float2 ge = *reinterpret_cast<const float2*>(gate + 64 + 8 * i);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          U[i][e] *= e & 1 ? be.y : be.x;
          V[i][e] = U[i][e] * (e & 1 ? ge.y : ge.x);
        }
      }
      put_tiles<3>(own + W::kW, w, V[0], V[1], lane);
      if constexpr (!SAVE) put_tiles<3>(own + W::kU, w, U[0], U[1], lane);
    }
    {
      uint32_t bk[4][DK / 64][4];
      float acc[DK / 32][4];
      load_rows<DK>(bk, sk, w, lane);
      const float last = reinterpret_cast<const float*>(st + W::kGate)[63];
      if (last == 0.f) zero(S);  // (what is not finite among it)
      team_bar(slice);
      // S <- e^{G_63} S + (e^{G_63 - G} U)^T K, this warp's columns
      outer_rows<DK>(acc, own + W::kW, bk, lane);
#pragma unroll
      for (int j = 0; j < DK / 32; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[j][e] = last * S[j][e] + acc[j][e];
      // every warp is past this chunk's
      put_state<DK, SAVE>(own, S, w, lane, snapshot(c + 1), row0, a.dv);
    }
    if constexpr (!SAVE) {
      // O += M U, this warp's tokens
      add_map_tokens(own + W::kU, se + 3 * kImage, w, lane, O);
    }
    const int n = min(kDeltaChunk, len - c * kDeltaChunk) - 16 * w;  // this warp's tokens, if any
    const int64_t orow = b * a.T + tok0 + int64_t(c) * kDeltaChunk + 16 * w;
    if (SAVE) continue;
    if (a.out_fp32) {
      float* out = static_cast<float*>(a.out);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 8 * i + t2 + e;
          if (r < n) {
            float* o = out + ((orow + r) * a.Hv + h) * a.dv + row0 + g4;
            o[0] = O[i][e];
            o[8] = O[i][2 + e];
          }
        }
    } else {
      // this warp's operand of X is no longer read: its place stages O
      store_tokens(O, own + W::kX + w * 3 * kOperand, static_cast<__nv_bfloat16*>(a.out) + (orow * a.Hv + h) * a.dv + row0,
                   int64_t(a.Hv) * a.dv, n, lane);
    }
  }
  if (a.state_out) store_state<DK>(S, a.state_out, srow, w, lane);
}

template <int DK, bool SAVE>
cudaError_t run_walk(const LaunchEnv& env, const WalkArgs& w) {
  using W = WalkShape<DK, SAVE>;
  const int ns = walk_slices(w.map.ndocs, w.Hv, w.dv, env.num_sms);
  const cudaError_t e = cudaFuncSetAttribute(delta_walk_kernel<DK, SAVE>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, W::smem(2));
  if (e != cudaSuccess) return e;
  return launch_pdl(delta_walk_kernel<DK, SAVE>,
                    dim3(unsigned(w.map.ndocs * w.Hv * (w.dv / (16 * ns)))),
                    dim3(kTeam * ns + 32),
                    W::smem(ns), env.stream, w);
}

// ---------------------------------------------------------------- recurrent
constexpr int kRecWarps = 4;
constexpr int kRecRows = 8;  // state rows a lane

template <typename T>
__device__ __forceinline__ float4 load4(const T* p, bool vec) {
  if constexpr (sizeof(T) == 4) {
    if (vec) return __ldg(reinterpret_cast<const float4*>(p));
    return make_float4(p[0], p[1], p[2], p[3]);
  } else {
    if (vec) {
      const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
      const float2 lo = unpack_bf16x2(u.x), hi = unpack_bf16x2(u.y);
      return make_float4(lo.x, lo.y, hi.x, hi.y);
    }
    return make_float4(__bfloat162float(p[0]), __bfloat162float(p[1]), __bfloat162float(p[2]),
                       __bfloat162float(p[3]));
  }
}
__device__ __forceinline__ float dot4(const float4& a, const float4& b) {
  return (a.x * b.x + a.y * b.y) + (a.z * b.z + a.w * b.w);
}

// A warp holds kRecRows * 128 / DK rows of the state, DK / 4 lanes a row, and
// walks the tokens.  S k and S q are taken together from the old state
// (o = scale (a S q + u k.q)), so the state is read once a token; the 16 sums
// a lane group needs are reduced by exchanging halves, 16 shuffles instead of
// 80.  For one token a sequence it is bound by reading and writing the state:
// 61 sequences of 20 heads of 128 x 128 in 23.5 us, 6.8 TB/s.
template <typename T, int DK>
__global__ void __launch_bounds__(32 * kRecWarps) delta_recurrent_kernel(DeltaArgs a) {
  constexpr int LPR = DK / 4;         // lanes a row
  constexpr int RPW = 32 / LPR;       // rows side by side
  constexpr int ROWS = kRecRows * RPW;  // rows a warp
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int slices = (a.dv + kRecWarps * ROWS - 1) / (kRecWarps * ROWS);
  const int h = (blockIdx.x / slices) % a.Hv, s = blockIdx.x / (slices * a.Hv);
  const int hk = h / (a.Hv / a.Hk);
  const int row0 = (int(blockIdx.x % slices) * kRecWarps + warp) * ROWS;
  const int col = 4 * (lane % LPR), sub = lane / LPR;
  griddep_wait();
  griddep_launch_dependents();
  if (row0 >= a.dv) return;
  // after the reduction the lane holds one sum: which (0: S k, 1: S q), of row `mine`
  const int idx = (lane >> (LPR == 32 ? 1 : 0)) & 15;
  const int mine = row0 + (idx & 7) * RPW + sub;
  const bool second = idx >= 8;
  const bool writer = second && (LPR == 16 || (lane & 1) == 0);
  const int64_t b = a.map.row(s);
  const int64_t t0 = a.map.start(s);
  const int len = a.map.len(s);
  int64_t pool_row = s;
  if (a.slots) {
    pool_row = load_id(a.slots, a.slots64, s);
    if (pool_row < 0 || pool_row >= a.pool) {  // no sequence here: a zero output
      if (writer && mine < a.dv)
        store_any(a.out, a.out_fp32, ((b * a.T + t0) * a.Hv + h) * a.dv + mine, 0.f);
      return;
    }
  }
  float4 S[kRecRows];
  const int64_t at = (pool_row * a.Hv + h) * int64_t(a.dv) * DK + col;
#pragma unroll
  for (int j = 0; j < kRecRows; ++j) {
    const int r = row0 + j * RPW + sub;
    S[j] = a.state_in && r < a.dv ? *reinterpret_cast<const float4*>(a.state_in + at + int64_t(r) * DK)
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const T* kp = static_cast<const T*>(a.k.data) + b * a.k.sb + t0 * a.k.st + hk * a.k.sh + col;
  const T* qp = static_cast<const T*>(a.q.data) + b * a.q.sb + t0 * a.q.st + hk * a.q.sh + col;
  const T* vp = static_cast<const T*>(a.v.data) + b * a.v.sb + t0 * a.v.st + h * a.v.sh + min(mine, a.dv - 1);
  const float* gp = a.g.data + b * a.g.sb + t0 * a.g.st + h * a.g.sh;
  const float* bp = a.beta.data + b * a.beta.sb + t0 * a.beta.st + h * a.beta.sh;
  float4 k, q;
  float v = 0.f, gt = 0.f, bt = 0.f;
  auto fetch = [&](int t) {
    k = load4<T>(kp + t * a.k.st, a.k.vec);
    q = load4<T>(qp + t * a.q.st, a.q.vec);
    v = load_any(vp, sizeof(T) == 4, t * a.v.st);
    gt = __ldg(gp + t * a.g.st);
    bt = __ldg(bp + t * a.beta.st);
  };
  if (len > 0) fetch(0);
  for (int t = 0; t < len; ++t) {
    const float4 kc = k, qc = q;
    const float vc = v, alpha = expf(gt), bc = bt;
    if (alpha == 0.f)  // clears a state that is not finite too
#pragma unroll
      for (int j = 0; j < kRecRows; ++j) S[j] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (t + 1 < len) fetch(t + 1);
    float x[16];
#pragma unroll
    for (int j = 0; j < kRecRows; ++j) {
      x[j] = dot4(S[j], kc);
      x[8 + j] = dot4(S[j], qc);
    }
    float kq = dot4(kc, qc);
#pragma unroll
    for (int m = LPR / 2; m; m >>= 1) kq += __shfl_xor_sync(~0u, kq, m);
    int m = LPR / 2;
#pragma unroll
    for (int cnt = 8; cnt; cnt >>= 1, m >>= 1) {
      const bool up = lane & m;
#pragma unroll
      for (int i = 0; i < cnt; ++i) {
        const float send = up ? x[i] : x[i + cnt], keep = up ? x[i + cnt] : x[i];
        x[i] = keep + __shfl_xor_sync(~0u, send, m);
      }
    }
    if constexpr (LPR == 32) x[0] += __shfl_xor_sync(~0u, x[0], 1);
    // both lanes of a pair learn S k and S q of the row
    const float other = __shfl_xor_sync(~0u, x[0], LPR / 2);
    const float sk = second ? other : x[0], sq = second ? x[0] : other;
    const float u = bc * (vc - alpha * sk);
    if (writer && mine < a.dv && a.out)
      store_any(a.out, a.out_fp32, ((b * a.T + t0 + t) * a.Hv + h) * a.dv + mine,
                a.scale * (alpha * sq + u * kq));
#pragma unroll
    for (int j = 0; j < kRecRows; ++j) {
      // u of row j lives where idx == j
      const float uj = __shfl_sync(~0u, u, (lane & ~(LPR - 1)) + (LPR == 32 ? 2 * j : j));
      S[j].x = alpha * S[j].x + uj * kc.x;
      S[j].y = alpha * S[j].y + uj * kc.y;
      S[j].z = alpha * S[j].z + uj * kc.z;
      S[j].w = alpha * S[j].w + uj * kc.w;
    }
  }
  if (a.state_out)
#pragma unroll
    for (int j = 0; j < kRecRows; ++j) {
      const int r = row0 + j * RPW + sub;
      if (r < a.dv) *reinterpret_cast<float4*>(a.state_out + at + int64_t(r) * DK) = S[j];
    }
}

template <typename T, int DK>
cudaError_t run_recurrent(const LaunchEnv& env, const DeltaArgs& a) {
  const int rows = kRecWarps * kRecRows * 128 / DK;
  const int64_t ctas = int64_t((a.dv + rows - 1) / rows) * a.Hv * a.map.ndocs;
  return launch_pdl(delta_recurrent_kernel<T, DK>, dim3(unsigned(ctas)), dim3(32 * kRecWarps), 0,
                    env.stream, a);
}

}  // namespace

cudaError_t launch_delta_prepare(const LaunchEnv& env, const DeltaArgs& a, unsigned char* blocks,
                                 bool grad, bool wide) {
  PrepArgs p;
  p.q = a.q;
  p.k = a.k;
  p.g = a.g;
  p.beta = a.beta;
  p.Hk = a.Hk;
  p.Hv = a.Hv;
  p.map = a.map;
  p.scale = a.scale;
  p.blocks = blocks;
  p.wide = wide;
  if (a.dk == 64) return grad ? run_prepare<64, true>(env, p) : run_prepare<64, false>(env, p);
  return grad ? run_prepare<128, true>(env, p) : run_prepare<128, false>(env, p);
}

// A team walks a slice of 16 rows, two to four slices an SM; a whole head an SM
// wins from the next round of slices on, unless it fills less than half of the
// tensor cores' 128 rows.  1024 tokens, heads of 128 x dv, us by slice / by head:
//   dv 128: 36 heads (288 slices) 78 / 84, 40 heads (320) 139 / 90
//   dv 64: 72 heads (288) 90 / 92, 80 heads (320) 152 / 100
//   dv 256: 16 heads (256) 74 / 78, 20 heads (320) 131 / 80
//   dv 32: 128 heads (256) 109 / 115, 160 heads (320) 174 / 180, 320 heads 281 / 289
// and the gradient alike (dv 128: 240 / 283, then 386 / 304; dv 32: 976 / 969).
bool delta_by_head(int64_t sequences, int Hv, int dv, int num_sms) {
  return dv > 32 && sequences * Hv * (dv / 16) > 2 * num_sms;
}

size_t delta_scratch(int64_t nchunks, int Hv) { return size_t(nchunks) * size_t(Hv) * kWideFwd; }

cudaError_t launch_team_walk(const LaunchEnv& env, const DeltaArgs& a, const unsigned char* blocks,
                             const DeltaSave* save) {
  WalkArgs w;
  w.q = a.q;
  w.k = a.k;
  w.v = a.v;
  w.Hk = a.Hk;
  w.Hv = a.Hv;
  w.dv = a.dv;
  w.T = a.T;
  w.map = a.map;
  w.scale = a.scale;
  w.state_in = a.state_in;
  w.state_out = a.state_out;
  w.out = a.out;
  w.out_fp32 = a.out_fp32;
  w.blocks = blocks;
  w.status = env.status;
  if (save) {
    w.save = *save;
    return a.dk == 64 ? run_walk<64, true>(env, w) : run_walk<128, true>(env, w);
  }
  return a.dk == 64 ? run_walk<64, false>(env, w) : run_walk<128, false>(env, w);
}

cudaError_t launch_delta_chunked(const LaunchEnv& env, const DeltaArgs& a) {
  const bool by_head = delta_by_head(a.map.ndocs, a.Hv, a.dv, env.num_sms);
  if (a.map.nchunks > 0) {
    const cudaError_t e = launch_delta_prepare(env, a, a.ws, false, by_head);
    if (e != cudaSuccess) return e;
  }
  return by_head ? launch_head_walk(env, a, a.ws, nullptr) : launch_team_walk(env, a, a.ws, nullptr);
}

cudaError_t launch_delta_recurrent(const LaunchEnv& env, const DeltaArgs& a) {
  if (a.fp32)
    return a.dk == 64 ? run_recurrent<float, 64>(env, a) : run_recurrent<float, 128>(env, a);
  return a.dk == 64 ? run_recurrent<__nv_bfloat16, 64>(env, a)
                    : run_recurrent<__nv_bfloat16, 128>(env, a);
}

}  // namespace ittt
