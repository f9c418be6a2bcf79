// k_delta_walk.cu -- the gated delta rule's walk over the chunks of a sequence,
// on tcgen05 with the state's products fed from tensor memory: up to 128 rows of a
// head an SM.  Sixteen warps hold the state in registers, four threads a row, and
// turn each product's accumulators into the next one's left operand (three bf16
// parts) in tensor memory; one warp issues the products, two load, one stores.
//
// A chunk is three links forward, four in the gradient's reverse walk, and what
// bounds it is their sum: 24 to 48 products of 64 columns (800 to 1600 cycles) and
// then 1000 to 2000 cycles in which the 16 warps read, scale, split and write, at
// 0.4 to 0.5 instructions a cycle and scheduler.  24001 tokens in 7 documents, 16
// heads of 64 x 128: 277 us, as long as its longest document of 6712, 5000 cycles a chunk;
// the gradient's walks of 2 x 4096 tokens, 20 heads of 128 x 128: 276 and 338 us,
// 8400 and 10200 cycles a chunk (measured on walks of 330 and 422 us, with snapshots
// in other parts: snapshots stored ahead of the products 45 and 30 us more; shared
// memory read through generic addresses, whose registers then spill, 43 and 20 more).
#include <algorithm>

#include "delta.cuh"

namespace ittt {
namespace {

// mma_ss with A in tensor memory: 128 rows of packed bf16 pairs.
__device__ __forceinline__ void mma_ts(uint32_t elected, uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo,
                                       uint32_t idesc, uint32_t accumulate) {
  constexpr uint32_t kHi = (1024u >> 4) | (1u << 14) | (2u << 29);
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 desc;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "setp.ne.b32 q, %6, 0;\n\t"
      "mov.b64 desc, {%2, %3};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], desc, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(kHi), "r"(idesc), "r"(accumulate), "r"(elected)
      : "memory");
}

template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// What follows from a and b is worked out anew: kept over the loop, some twenty
// addresses cost registers, and with 227 KB of shared memory in use there is
// hardly an L1 left for what is spilled.
__device__ __forceinline__ void again(int& a, int& b) { asm volatile("" : "+r"(a), "+r"(b)); }

// 16 numbers of this thread's row as operand columns: NP parts, `part` columns
// from one to the next.
template <int NP>
__device__ __forceinline__ void put16(uint32_t taddr, uint32_t part, const float* v) {
  uint32_t r[NP][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t p[NP];
    split2<NP>(v[2 * i], v[2 * i + 1], p);
#pragma unroll
    for (int q = 0; q < NP; ++q) r[q][i] = p[q];
  }
#pragma unroll
  for (int q = 0; q < NP; ++q)
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(
                     taddr + q * part),
                 "r"(r[q][0]), "r"(r[q][1]), "r"(r[q][2]), "r"(r[q][3]), "r"(r[q][4]), "r"(r[q][5]),
                 "r"(r[q][6]), "r"(r[q][7])
                 : "memory");
}

constexpr int kTokTile = 16384;  // [128 rows of dv][64 tokens] bf16, pieces of 8 swizzled

// A quarter of a row of a state into a snapshot.
template <int DK>
__device__ __forceinline__ void snap_parts(unsigned char* snap, int dv, int row, int quarter, const float* S) {
#pragma unroll
  for (int i = 0; i < DK / 4; i += 8) {
    uint32_t p[4][3];
#pragma unroll
    for (int j = 0; j < 4; ++j) split2<3>(S[i + 2 * j], S[i + 2 * j + 1], p[j]);
    unsigned char* at = snap + piece_at<DK>(dv, row, 0, (quarter * (DK / 4) + i) / 8);
    const int64_t part = int64_t(DK / 8) * min(kPanel, dv - row / kPanel * kPanel) * 16;
#pragma unroll
    for (int q = 0; q < 3; ++q)
      *reinterpret_cast<uint4*>(at + q * part) = make_uint4(p[0][q], p[1][q], p[2][q], p[3][q]);
  }
}
// 16 numbers of row r, three parts, as pieces of three tiles of 128 rows.
__device__ __forceinline__ void stage_parts(unsigned char* tiles, int r, int piece, const float* v) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t p[4][3];
#pragma unroll
    for (int j = 0; j < 4; ++j) split2<3>(v[8 * i + 2 * j], v[8 * i + 2 * j + 1], p[j]);
#pragma unroll
    for (int q = 0; q < 3; ++q)
      *reinterpret_cast<uint4*>(tiles + q * kTokTile + tile_at<8>(r, piece + i)) =
          make_uint4(p[0][q], p[1][q], p[2][q], p[3][q]);
  }
}

struct TcArgs {
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
  DeltaSave save;  // kSaved only
};

constexpr int kTcWarps = 16;  // compute warps: four threads a row of the state
constexpr int kTcThreads = 32 * (kTcWarps + 4);
constexpr int kTok = kDeltaChunk / 4;  // tokens a thread
// Registers a thread: 96 at launch, split between the warpgroups that hold the
// state and the one that serves them (512 x 104 + 128 x 64 = 640 x 96).
constexpr int kTcMore = 104, kTcFewer = 64;

// A [64 tokens][up to 128 dv] block by one warp, plain rows of 256 bytes.  (A bulk
// copy a row costs the copy engine some 70 cycles, and a chunk has two or three
// such blocks: 64 rows took 4000 to 6000 cycles either way.)
__device__ __forceinline__ void load_rows(unsigned char* dst, const __nv_bfloat16* src, int64_t st, int pieces, int n,
                                          bool vec, int lane) {
  const int c = lane & 15, r0 = lane >> 4;
  if (c >= pieces) return;
  const __nv_bfloat16* p = src + r0 * st + c * 8;
  unsigned char* d = dst + lane * 16;
  if (vec) {
    const uint32_t to = smem_u32(d);
#pragma unroll 8
    for (int r = r0, i = 0; i < 32; ++i, r += 2, p += 2 * st) cp16(to + i * 512, r < n ? p : src, r < n);
  } else {
    for (int r = r0; r < kDeltaChunk; r += 2, p += 2 * st, d += 512) {
      if (r < n)
        store_piece(d, p);
      else
        *reinterpret_cast<uint4*>(d) = make_uint4(0, 0, 0, 0);
    }
  }
}
// The first n rows of such a block to memory.
__device__ __forceinline__ void store_rows(__nv_bfloat16* dst, int64_t st, const unsigned char* src, int pieces, int n,
                                           int lane) {
  const int c = lane & 15, r0 = lane >> 4;
  if (c >= pieces) return;
  __nv_bfloat16* p = dst + r0 * st + c * 8;
#pragma unroll 8
  for (int r = r0; r < n; r += 2, p += 2 * st) *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(src + r * 256 + c * 16);
}

// out_ready: one a stage, since a stage's next phase waits for the storing warp to
// have released it; with one for both, the chunk after could complete its phase
// before that warp looks, and a wait by parity would miss both.
struct TcBars {
  uint64_t full[2], empty[2], out_ready[2], out_free;
  uint64_t s_ready, x_ready, w_ready, u_ready;         // operands in tensor memory
  uint64_t p_done, q_done, e_done, d_done, m_done;     // products
  uint32_t tmem;
  int abort;
};

// Columns of tensor memory.  The state's three parts (64 columns each at dk 128)
// give way to those of W and U once both products with them are done; U's
// product with the scores takes the place of X's parts, Q S^T that of the
// state's update.
constexpr uint32_t kTmS = 0, kTmW = 0, kTmU = 96, kTmX = 192, kTmO = 192, kTmP = 288, kTmD = 352;

// Shared memory: two stages of what the products read (K, E map, for the output Q and
// the scores) and of V and the gates, then what leaves: the output in bf16, or E in
// three parts.
enum HeadOut { kOutBf16, kOutFp32, kSaved };  // what leaves; kSaved: the gradient's forward pass
template <int DK, HeadOut OUT>
struct TcShape {
  static constexpr uint32_t kTile = kDeltaChunk * DK * 2;
  static constexpr uint32_t kQ = kTile, kE = (OUT == kSaved ? 1 : 2) * kTile, kM = kE + 3 * kWideTile;
  static constexpr uint32_t kTiles = kM + (OUT == kSaved ? 0 : 3 * kWideTile);  // what the products read
  static constexpr uint32_t kV = 0, kGate = kDeltaChunk * 256, kRest = kGate + 768;
  static constexpr uint32_t kOut = 2 * kTiles + 2 * kRest;
  static constexpr uint32_t kBars = kOut + (OUT == kSaved ? 3 * kTokTile : OUT == kOutBf16 ? kDeltaChunk * 256 : 0);
  static constexpr int64_t kBlock = OUT == kSaved ? kWideGrad : kWideFwd;
  static constexpr uint32_t kSmem = kBars + sizeof(TcBars) + 1024;
};

template <int DK, HeadOut OUT>
__global__ void __launch_bounds__(kTcThreads, 1) head_walk_kernel(TcArgs a) {
  extern __shared__ unsigned char smem_raw[];
  using W = TcShape<DK, OUT>;
  constexpr bool SAVE = OUT == kSaved;
  constexpr int HS = DK / 4;  // columns of the state a thread
  constexpr uint32_t SP = DK / 2;  // columns of tensor memory a part of the state
  unsigned char* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);  // an offset: its loads stay shared ones
  TcBars* bars = reinterpret_cast<TcBars*>(smem + W::kBars);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->full[i], 3);
      mbar_init(&bars->empty[i], kTcWarps + 1);
    }
    uint64_t* ready[] = {&bars->s_ready, &bars->x_ready, &bars->w_ready, &bars->u_ready};
    for (uint64_t* r : ready) mbar_init(r, kTcWarps);
    for (int i = 0; i < 2; ++i) mbar_init(&bars->out_ready[i], kTcWarps);
    mbar_init(&bars->out_free, 1);
    uint64_t* done[] = {&bars->p_done, &bars->q_done, &bars->e_done, &bars->d_done, &bars->m_done};
    for (uint64_t* d : done) mbar_init(d, 1);
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == kTcWarps) {
    tmem_alloc(&bars->tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tm = bars->tmem;
  griddep_wait();
  griddep_launch_dependents();
  const int panels = (a.dv + 127) / 128;
  const int h = (blockIdx.x / panels) % a.Hv, s = blockIdx.x / (panels * a.Hv);
  const int row0 = (blockIdx.x % panels) * 128, rows = min(128, a.dv - row0);
  const int64_t b = a.map.row(s), tok0 = a.map.start(s);
  const int len = a.map.len(s), nchunks = (len + kDeltaChunk - 1) / kDeltaChunk;
  const int64_t chunk0 = a.map.chunk0(s);
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (!mbar_wait(bar, parity, &bars->abort)) raise_abort(&bars->abort, a.status, kStatusTimeout);
  };

  if (warp >= kTcWarps) fewer_registers<kTcFewer>();
  if (warp > kTcWarps) {
    // ------------------------------------- the loaders, and the output's stores
    const int hk = h / (a.Hv / a.Hk), lw = warp - kTcWarps - 1;  // 0 .. 2
    const int pieces = rows / 8;
    if (lw == 2 && SAVE) {
      unsigned char* e = a.save.e + (chunk0 * a.Hv + h) * token_tiles(a.dv) + row0 * 128;
      for (int c = 0; c < nchunks; ++c, e += a.Hv * token_tiles(a.dv)) {
        wait(&bars->out_ready[c & 1], (c >> 1) & 1);
        if (lane == 0) {
          for (int p = 0; p < 3; ++p) bulk_store(e + int64_t(p) * a.dv * 128, smem + W::kOut + p * kTokTile, rows * 128);
          bulk_commit_group();
          bulk_wait_group_read<0>();
          mbar_arrive(&bars->out_free);
        }
        __syncwarp();
      }
      bulk_wait_group_all();
    } else if (lw == 2 && OUT == kOutBf16) {
      auto* out = static_cast<__nv_bfloat16*>(a.out) + ((b * a.T + tok0) * a.Hv + h) * a.dv + row0;
      const int64_t step = int64_t(a.Hv) * a.dv;
      for (int c = 0; c < nchunks; ++c, out += kDeltaChunk * step) {
        wait(&bars->out_ready[c & 1], (c >> 1) & 1);
        store_rows(out, step, smem + W::kOut, pieces, min(kDeltaChunk, len - c * kDeltaChunk), lane);
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->out_free);
      }
    } else if (lw < 2) {
      // K and V, Q; in the gradient's form K, V
      const bool tiles_here = !SAVE || lw == 0, rows_here = lw == (SAVE ? 1 : 0);
      const HeadView& tv = lw ? a.q : a.k;
      const auto* tile = static_cast<const __nv_bfloat16*>(tv.data) + b * tv.sb + tok0 * tv.st + hk * tv.sh;
      const auto* plain = static_cast<const __nv_bfloat16*>(a.v.data) + b * a.v.sb + tok0 * a.v.st + h * a.v.sh + row0;
      const int64_t tile_st = tv.st, plain_st = a.v.st;
      const bool tile_vec = tv.vec, plain_vec = a.v.vec;
      for (int c = 0; c < nchunks; ++c, tile += kDeltaChunk * tile_st, plain += kDeltaChunk * plain_st) {
        const int st = c & 1, n = min(kDeltaChunk, len - c * kDeltaChunk);
        if (c >= 2) wait(&bars->empty[st], ((c >> 1) & 1) ^ 1);
        if (__any_sync(~0u, aborted(&bars->abort))) break;
        unsigned char* tiles = smem + st * W::kTiles;
        unsigned char* rest = smem + 2 * W::kTiles + st * W::kRest;
        if (lw == 0 && lane == 0) {
          const unsigned char* blk = a.blocks + ((chunk0 + c) * a.Hv + h) * W::kBlock;
          mbar_arrive_expect_tx(&bars->full[st], (SAVE ? 3 : 6) * kWideTile + 768);
          bulk_load(tiles + W::kE, blk, (SAVE ? 3 : 6) * kWideTile, &bars->full[st]);
          bulk_load(rest + W::kGate, blk + kWideGate, 768, &bars->full[st]);
        }
        __syncwarp();
        if (tiles_here)
#pragma unroll
          for (int i = 0; i < DK / 64; ++i)
            warp_load_tile<8>(tiles + lw * W::kQ + i * 8192, tile + 64 * i, tile_st, n, tile_vec, lane);
        if (rows_here) load_rows(rest + W::kV, plain, plain_st, pieces, n, plain_vec, lane);
        cp_wait_all();
        fence_proxy_async_smem();  // K and Q are read by the tensor cores
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->full[st]);
      }
    }
  } else if (warp == kTcWarps) {
    // ----------------------------------------------------------- the products
    const uint32_t on = elect_one();
    uint32_t tmu = __shfl_sync(~0u, tm, 0);
    const uint32_t base = __shfl_sync(~0u, smem_u32(smem), 0) >> 4;
    constexpr uint32_t id_tok = idesc_bf16_f32(128, 64, false, false);
    constexpr uint32_t id_state = idesc_bf16_f32(128, DK, false, true);
    constexpr uint32_t lbo = (8192u >> 4) << 16;
    for (int c = 0; c < nchunks; ++c) {
      const int st = c & 1;
      const uint32_t par = c & 1, sk = base + st * (W::kTiles >> 4);
      asm volatile("" : "+r"(tmu));  // operand addresses are not kept, as by again()
      // a triangular map's product with the parts at `x`, small terms first;
      // tokens before a step's do not see it
      auto map = [&](uint32_t d, uint32_t x, uint32_t tile) {
#pragma unroll
        for (int sum = 2; sum >= 0; --sum)
#pragma unroll
          for (int p = 0; p <= sum; ++p)
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              mma_ts(on, d + 16 * ks, x + p * 32 + ks * 8,
                     tile + (((sum - p) * kWideTile + ks * (16 * 128 + 32)) >> 4),
                     idesc_bf16_f32(128, 64 - 16 * ks, false, false), sum < 2 || p > 0 || ks > 0);
      };
      wait(&bars->full[st], (c >> 1) & 1);
      wait(&bars->s_ready, par);
      tc_fence_after_sync();
#pragma unroll
      for (int p = 2; p >= 0; --p)
#pragma unroll
        for (int ks = 0; ks < DK / 16; ++ks)
          mma_ts(on, tmu + kTmP, tmu + kTmS + p * SP + ks * 8, sk + (((ks >> 2) * 8192 + (ks & 3) * 32) >> 4), id_tok,
                 p < 2 || ks > 0);
      commit(on, &bars->p_done);
      if constexpr (!SAVE) {
#pragma unroll
        for (int p = 2; p >= 0; --p)
#pragma unroll
          for (int ks = 0; ks < DK / 16; ++ks)
            mma_ts(on, tmu + kTmD, tmu + kTmS + p * SP + ks * 8,
                   sk + ((W::kQ + (ks >> 2) * 8192 + (ks & 3) * 32) >> 4), id_tok, p < 2 || ks > 0);
        commit(on, &bars->q_done);
      }
      wait(&bars->x_ready, par);
      tc_fence_after_sync();
      map(tmu + kTmP, tmu + kTmX, sk + (W::kE >> 4));
      commit(on, &bars->e_done);
      wait(&bars->w_ready, par);
      tc_fence_after_sync();
#pragma unroll
      for (int p = 2; p >= 0; --p)
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          mma_ts(on, tmu + kTmD, tmu + kTmW + p * 32 + ks * 8, sk + lbo + ((ks * 2048) >> 4), id_state, p < 2 || ks > 0);
      commit(on, &bars->d_done);
      if constexpr (!SAVE) {
        wait(&bars->u_ready, par);
        tc_fence_after_sync();
        map(tmu + kTmO, tmu + kTmU, sk + (W::kM >> 4));
        commit(on, &bars->m_done);
      }
      commit(on, &bars->empty[st]);
    }
    __syncwarp();
  } else if (warp < kTcWarps) {
    more_registers<kTcMore>();
    // -------------------------------------------------------------- the state
    int row = (warp & 3) * 32 + lane, quarter = warp >> 2;
    const bool active = row < rows;
    const uint32_t trow = tm + (uint32_t((warp & 3) * 32) << 16);
    float S[HS], O[kTok];
    const int64_t srow = ((int64_t(s) * a.Hv + h) * a.dv + row0 + row) * DK + quarter * HS;
#pragma unroll
    for (int i = 0; i < HS; i += 4) {
      const float4 v = active && a.state_in ? *reinterpret_cast<const float4*>(a.state_in + srow + i)
                                            : make_float4(0.f, 0.f, 0.f, 0.f);
      S[i] = v.x;
      S[i + 1] = v.y;
      S[i + 2] = v.z;
      S[i + 3] = v.w;
    }
    auto arrive = [&](uint64_t* bar) {
      tmem_wait_st();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    float last = 1.f;
    // chunk c's update of S and its output, which the next chunk's first product
    // runs beside
    auto finish_state = [&](int c) {
      wait(&bars->d_done, c & 1);
      tc_fence_after_sync();
#pragma unroll
      for (int i = 0; i < HS; i += 16) {
        float v[16];
        read16(trow + kTmD + quarter * HS + i, v);
#pragma unroll
        for (int e = 0; e < 16; ++e) S[i + e] = last * S[i + e] + v[e];
      }
      if constexpr (!SAVE) {
        wait(&bars->m_done, c & 1);
        tc_fence_after_sync();
        float v[kTok];
        read16(trow + kTmO + kTok * quarter, v);
#pragma unroll
        for (int e = 0; e < kTok; ++e) O[e] += v[e];
      }
    };
    auto finish_out = [&](int c) {
      if constexpr (OUT == kOutBf16) {
        if (c > 0) wait(&bars->out_free, (c - 1) & 1);
        unsigned char* to = smem + W::kOut + kTok * quarter * 256 + row * 2;
#pragma unroll
        for (int e = 0; e < kTok; ++e) *reinterpret_cast<__nv_bfloat16*>(to + e * 256) = __float2bfloat16_rn(O[e]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->out_ready[c & 1]);
      } else if constexpr (OUT == kOutFp32) {
        const int n = min(kDeltaChunk, len - c * kDeltaChunk) - kTok * quarter;
        float* out = static_cast<float*>(a.out) +
                     ((b * a.T + tok0 + int64_t(c) * kDeltaChunk + kTok * quarter) * a.Hv + h) * a.dv + row0 + row;
        const int64_t step = int64_t(a.Hv) * a.dv;
        if (active)
#pragma unroll
          for (int e = 0; e < kTok; ++e)
            if (e < n) out[e * step] = O[e];
      }
    };
    // the state as the next product's operand
    auto put_s = [&]() {
#pragma unroll
      for (int i = 0; i < HS; i += 16) put16<3>(trow + kTmS + (quarter * HS + i) / 2, SP, S + i);
    };
    // its snapshot, beside the products: split again, since the stores take twice as
    // long as the operand (between put and arrive they cost every chunk 2000 cycles)
    auto snap_s = [&](int c) {
      if (active)
        snap_parts<DK>(a.save.snap + ((chunk0 + c) * a.Hv + h) * state_parts(a.dv, DK), a.dv, row0 + row, quarter, S);
    };
    for (int c = 0; c < nchunks; ++c) {
      const int st = c & 1;
      const uint32_t par = c & 1;
      again(row, quarter);
      if (c > 0) finish_state(c - 1);
      const unsigned char* rest = smem + 2 * W::kTiles + st * W::kRest;
      put_s();
      arrive(&bars->s_ready);
      if constexpr (SAVE) snap_s(c);
      if (c > 0) finish_out(c - 1);
      const float4* gate = reinterpret_cast<const float4*>(rest + W::kGate) + quarter * (kTok / 4);
      const unsigned char* vcol = rest + W::kV + kTok * quarter * 256 + row * 2;
      float x[kTok];
      __nv_bfloat16 v[kTok];
      wait(&bars->full[st], (c >> 1) & 1);
      const bool reset = *reinterpret_cast<const float*>(rest + W::kGate) == 0.f;  // clears what is not finite too
#pragma unroll
      for (int e = 0; e < kTok; ++e) v[e] = *reinterpret_cast<const __nv_bfloat16*>(vcol + e * 256);
      wait(&bars->p_done, par);
      tc_fence_after_sync();
      // X = V - e^G (K S^T)
      read16(trow + kTmP + kTok * quarter, x);
      if (reset) {
#pragma unroll
        for (int i = 0; i < HS; ++i) S[i] = 0.f;
#pragma unroll
        for (int e = 0; e < kTok; ++e) x[e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < kTok; e += 4) {
        const float4 eg = gate[e / 4];
        const float g4[4] = {eg.x, eg.y, eg.z, eg.w};
#pragma unroll
        for (int f = 0; f < 4; ++f) x[e + f] = (active ? __bfloat162float(v[e + f]) : 0.f) - g4[f] * x[e + f];
      }
      put16<3>(trow + kTmX + kTok / 2 * quarter, 32, x);
      arrive(&bars->x_ready);
      if constexpr (!SAVE) {
        wait(&bars->q_done, par);
        tc_fence_after_sync();
        read16(trow + kTmD + kTok * quarter, O);
#pragma unroll
        for (int e = 0; e < kTok; e += 4) {
          const float4 eg = gate[e / 4];
          O[e] *= a.scale * eg.x;
          O[e + 1] *= a.scale * eg.y;
          O[e + 2] *= a.scale * eg.z;
          O[e + 3] *= a.scale * eg.w;
        }
        if (reset)
#pragma unroll
          for (int e = 0; e < kTok; ++e) O[e] = 0.f;
      }
      float ge[kTok];
#pragma unroll
      for (int e = 0; e < kTok; e += 4) {
        const float4 g2 = gate[16 + e / 4];
        ge[e] = g2.x;
        ge[e + 1] = g2.y;
        ge[e + 2] = g2.z;
        ge[e + 3] = g2.w;
      }
      last = reinterpret_cast<const float*>(rest + W::kGate)[63];
      wait(&bars->e_done, par);
      tc_fence_after_sync();
      // W = e^{G_63 - G} U first, which the state waits for; U = b E
      read16(trow + kTmP + kTok * quarter, x);
#pragma unroll
      for (int e = 0; e < kTok; e += 4) {
        const float4 be = gate[32 + e / 4];
        ge[e] *= be.x * x[e];
        ge[e + 1] *= be.y * x[e + 1];
        ge[e + 2] *= be.z * x[e + 2];
        ge[e + 3] *= be.w * x[e + 3];
      }
      put16<3>(trow + kTmW + kTok / 2 * quarter, 32, ge);
      arrive(&bars->w_ready);
      if constexpr (SAVE) {
        if (lane == 0) mbar_arrive(&bars->empty[st]);  // V and the gates are read
        // E's parts leave
        if (c > 0) wait(&bars->out_free, (c - 1) & 1);
        stage_parts(smem + W::kOut, row, 2 * quarter, x);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->out_ready[st]);
      } else {
#pragma unroll
        for (int e = 0; e < kTok; e += 4) {
          const float4 be = gate[32 + e / 4];
          x[e] *= be.x;
          x[e + 1] *= be.y;
          x[e + 2] *= be.z;
          x[e + 3] *= be.w;
        }
        put16<3>(trow + kTmU + kTok / 2 * quarter, 32, x);
        arrive(&bars->u_ready);
        if (lane == 0) mbar_arrive(&bars->empty[st]);  // V and the gates are read
      }
    }
    if (nchunks > 0) {
      finish_state(nchunks - 1);
      finish_out(nchunks - 1);
    }
    if (active && a.state_out)
#pragma unroll
      for (int i = 0; i < HS; i += 4)
        *reinterpret_cast<float4*>(a.state_out + srow + i) = make_float4(S[i], S[i + 1], S[i + 2], S[i + 3]);
    tc_fence_before_sync();
  }
  settle(&bars->abort);
  __syncthreads();
  tc_fence_after_sync();
  if (warp == kTcWarps) tmem_dealloc(tm, 512);
}

// ------------------------------------------------------------------ reverse
// Shared memory: two stages of what the products read (K, Q, scores, R map, dO; dR's
// parts leave from the place of the scores and the map), of dV on its way out, and of
// the gates.
template <int DK>
struct BackShape {
  static constexpr uint32_t kTile = kDeltaChunk * DK * 2;
  static constexpr uint32_t kQ = kTile, kM = 2 * kTile, kR = kM + 3 * kWideTile, kDo = kR + 3 * kWideTile;
  static constexpr uint32_t kTiles = kDo + 2 * kWideTile;
  static constexpr uint32_t kV = 0, kGate = kDeltaChunk * 256, kRest = kGate + 768;
  static constexpr uint32_t kBars = 2 * kTiles + 2 * kRest;
  static constexpr uint32_t kSmem = kBars + sizeof(TcBars) + 1024;
};
// Tensor memory as in the forward walk; the parts of scale e^G dO take U's place,
// M^T dO that of Q S^T.
constexpr uint32_t kTmY = 96;
// (e^G dX)^T K has an accumulator of its own, over X's parts and dR, which are read by
// then: added to the other product's full-size sum, each step's rounding towards zero
// is one more of the sum's last place (the starting states' gradient was off by 4.8e-7
// in the Frobenius norm, 1.5e-7 now), and the two need not wait for one another (375 us, 338 now).
constexpr uint32_t kTmE = 192;

// The reverse walk of a head, with dS in the state's place.
template <int DK>
__global__ void __launch_bounds__(kTcThreads, 1) head_reverse_kernel(ReverseArgs a) {
  extern __shared__ unsigned char smem_raw[];
  using W = BackShape<DK>;
  constexpr int HS = DK / 4;
  constexpr uint32_t SP = DK / 2;
  unsigned char* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);  // an offset: its loads stay shared ones
  TcBars* bars = reinterpret_cast<TcBars*>(smem + W::kBars);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->full[i], 3);
      mbar_init(&bars->empty[i], kTcWarps + 2);
    }
    uint64_t* ready[] = {&bars->s_ready, &bars->x_ready, &bars->w_ready, &bars->u_ready, &bars->out_ready[0], &bars->out_ready[1]};
    for (uint64_t* r : ready) mbar_init(r, kTcWarps);
    uint64_t* done[] = {&bars->p_done, &bars->q_done, &bars->e_done, &bars->d_done};
    for (uint64_t* d : done) mbar_init(d, 1);
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == kTcWarps) {
    tmem_alloc(&bars->tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tm = bars->tmem;
  griddep_wait();
  griddep_launch_dependents();
  const int panels = (a.dv + 127) / 128;
  const int h = (blockIdx.x / panels) % a.Hv, s = blockIdx.x / (panels * a.Hv);
  const int row0 = (blockIdx.x % panels) * 128, rows = min(128, a.dv - row0);
  const int64_t b = a.map.row(s), tok0 = a.map.start(s);
  const int len = a.map.len(s), nchunks = (len + kDeltaChunk - 1) / kDeltaChunk;
  const int64_t chunk0 = a.map.chunk0(s);
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (!mbar_wait(bar, parity, &bars->abort)) raise_abort(&bars->abort, a.status, kStatusTimeout);
  };

  if (warp >= kTcWarps) fewer_registers<kTcFewer>();
  if (warp > kTcWarps) {
    // ------------------------------------------- the loaders, and dV's stores
    const int hk = h / (a.Hv / a.Hk), lw = warp - kTcWarps - 1;
    const int pieces = rows / 8;
    if (lw == 2) {
      const int64_t step = int64_t(a.Hv) * a.dv, c0 = int64_t(nchunks - 1) * kDeltaChunk;
      auto* out = a.dvp + ((b * a.T + tok0 + c0) * a.Hv + h) * a.dv + row0;
      for (int it = 0; it < nchunks; ++it, out -= kDeltaChunk * step) {
        const int c = nchunks - 1 - it, st = it & 1;
        wait(&bars->out_ready[st], (it >> 1) & 1);
        if (lane < 3)
          bulk_store(a.dr + ((chunk0 + c) * a.Hv + h) * token_tiles(a.dv) + (int64_t(lane) * a.dv + row0) * 128,
                     smem + st * W::kTiles + W::kM + lane * kTokTile, rows * 128);
        bulk_commit_group();
        store_rows(out, step, smem + 2 * W::kTiles + st * W::kRest + W::kV, pieces,
                   min(kDeltaChunk, len - c * kDeltaChunk), lane);
        bulk_wait_group_read<0>();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->empty[st]);
      }
      bulk_wait_group_all();
    } else {
      // K and half of dO; Q and the other half
      const HeadView& tv = lw ? a.q : a.k;
      const int64_t t = tok0 + int64_t(nchunks - 1) * kDeltaChunk;
      const auto* tile = static_cast<const __nv_bfloat16*>(tv.data) + b * tv.sb + t * tv.st + hk * tv.sh;
      const auto* dop = static_cast<const __nv_bfloat16*>(a.dout.data) + b * a.dout.sb + t * a.dout.st + h * a.dout.sh +
                        row0 + 64 * lw;
      const int64_t tile_st = tv.st;
      const bool tile_vec = tv.vec;
      for (int it = 0; it < nchunks; ++it) {
        const int c = nchunks - 1 - it, st = it & 1, n = min(kDeltaChunk, len - c * kDeltaChunk);
        unsigned char* tiles = smem + st * W::kTiles;
        unsigned char* rest = smem + 2 * W::kTiles + st * W::kRest;
        if (it >= 2) wait(&bars->empty[st], ((it >> 1) & 1) ^ 1);
        if (__any_sync(~0u, aborted(&bars->abort))) break;
        if (lw == 0 && lane == 0) {
          const unsigned char* blk = a.blocks + ((chunk0 + c) * a.Hv + h) * int64_t(kWideGrad);
          mbar_arrive_expect_tx(&bars->full[st], 6 * kWideTile + 768);
          bulk_load(tiles + W::kM, blk + kWideM, 3 * kWideTile, &bars->full[st]);
          bulk_load(tiles + W::kR, blk + kWideR, 3 * kWideTile, &bars->full[st]);
          bulk_load(rest + W::kGate, blk + kWideGate, 768, &bars->full[st]);
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < DK / 64; ++i)
          warp_load_tile<8>(tiles + lw * W::kQ + i * 8192, tile + 64 * i, tile_st, n, tile_vec, lane);
        // dO as a left operand: rows along the sum over tokens; columns past the
        // head's are zero
        warp_load_tile<8>(tiles + W::kDo + lw * kWideTile, dop, a.dout.st, n, a.dout.vec, lane, pieces - 8 * lw);
        cp_wait_all();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->full[st]);
        tile -= kDeltaChunk * tile_st;
        dop -= kDeltaChunk * a.dout.st;
      }
    }
  } else if (warp == kTcWarps) {
    // ----------------------------------------------------------- the products
    const uint32_t on = elect_one();
    uint32_t tmu = __shfl_sync(~0u, tm, 0);
    const uint32_t base = __shfl_sync(~0u, smem_u32(smem), 0) >> 4;
    constexpr uint32_t id_tok = idesc_bf16_f32(128, 64, false, false);
    constexpr uint32_t id_state = idesc_bf16_f32(128, DK, false, true);
    constexpr uint32_t lbo = (8192u >> 4) << 16;
    for (int it = 0; it < nchunks; ++it) {
      const int st = it & 1;
      const uint32_t par = it & 1, sk = base + st * (W::kTiles >> 4);
      asm volatile("" : "+r"(tmu));  // operand addresses are not kept, as by again()
      wait(&bars->full[st], (it >> 1) & 1);
      wait(&bars->s_ready, par);
      tc_fence_after_sync();
      // K dS'^T
#pragma unroll
      for (int p = 2; p >= 0; --p)
#pragma unroll
        for (int ks = 0; ks < DK / 16; ++ks)
          mma_ts(on, tmu + kTmP, tmu + kTmS + p * SP + ks * 8, sk + (((ks >> 2) * 8192 + (ks & 3) * 32) >> 4), id_tok,
                 p < 2 || ks > 0);
      commit(on, &bars->p_done);
      // M^T dO: a step's tokens see the tokens up to their own
#pragma unroll
      for (int p = 2; p >= 0; --p)
#pragma unroll
        for (int ks = 3; ks >= 0; --ks)
          mma_ss(on, tmu + kTmD, sk + lbo + ((W::kDo + ks * 2048) >> 4), sk + ((W::kM + p * kWideTile + ks * 2048) >> 4),
                 idesc_bf16_f32(128, 16 * (ks + 1), true, true), p < 2 || ks < 3);
      commit(on, &bars->q_done);
      wait(&bars->x_ready, par);
      tc_fence_after_sync();
      // dU0 R
#pragma unroll
      for (int sum = 2; sum >= 0; --sum)
#pragma unroll
        for (int p = 0; p <= sum; ++p)
#pragma unroll
          for (int ks = 3; ks >= 0; --ks)
            mma_ts(on, tmu + kTmP, tmu + kTmX + p * 32 + ks * 8, sk + ((W::kR + (sum - p) * kWideTile + ks * 2048) >> 4),
                   idesc_bf16_f32(128, 16 * (ks + 1), false, true), sum < 2 || p > 0 || ks < 3);
      commit(on, &bars->e_done);
      wait(&bars->u_ready, par);
      tc_fence_after_sync();
      // (scale e^G dO)^T Q
#pragma unroll
      for (int p = 2; p >= 0; --p)
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          mma_ts(on, tmu + kTmD, tmu + kTmY + p * 32 + ks * 8, sk + lbo + ((W::kQ + ks * 2048) >> 4), id_state,
                 p < 2 || ks > 0);
      wait(&bars->w_ready, par);
      tc_fence_after_sync();
      // - (e^G dX)^T K
#pragma unroll
      for (int p = 2; p >= 0; --p)
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          mma_ts(on, tmu + kTmE, tmu + kTmW + p * 32 + ks * 8, sk + lbo + ((ks * 2048) >> 4), id_state, p < 2 || ks > 0);
      commit(on, &bars->d_done);
      commit(on, &bars->empty[st]);
    }
    __syncwarp();
  } else if (warp < kTcWarps) {
    more_registers<kTcMore>();
    int row = (warp & 3) * 32 + lane, quarter = warp >> 2;
    const bool active = row < rows;
    const uint32_t trow = tm + (uint32_t((warp & 3) * 32) << 16);
    float S[HS];  // dS'
    const int64_t srow = ((int64_t(s) * a.Hv + h) * a.dv + row0 + row) * DK + quarter * HS;
#pragma unroll
    for (int i = 0; i < HS; i += 4) {
      const float4 v = active && a.dstate_out ? *reinterpret_cast<const float4*>(a.dstate_out + srow + i)
                                              : make_float4(0.f, 0.f, 0.f, 0.f);
      S[i] = v.x;
      S[i + 1] = v.y;
      S[i + 2] = v.z;
      S[i + 3] = v.w;
    }
    auto arrive = [&](uint64_t* bar) {
      tmem_wait_st();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    for (int it = 0; it < nchunks; ++it) {
      const int c = nchunks - 1 - it, st = it & 1;
      const uint32_t par = it & 1;
      again(row, quarter);
      const int64_t ch = (chunk0 + c) * a.Hv + h;
#pragma unroll
      for (int i = 0; i < HS; i += 16) put16<3>(trow + kTmS + (quarter * HS + i) / 2, SP, S + i);
      arrive(&bars->s_ready);
      if (active) snap_parts<DK>(a.dsnap + ch * state_parts(a.dv, DK), a.dv, row0 + row, quarter, S);
      unsigned char* tiles = smem + st * W::kTiles;
      unsigned char* rest = smem + 2 * W::kTiles + st * W::kRest;
      const float4* gate = reinterpret_cast<const float4*>(rest + W::kGate) + quarter * (kTok / 4);
      float x[kTok], y[kTok];
      wait(&bars->full[st], (it >> 1) & 1);
      {
        const unsigned char* col = tiles + W::kDo + (row >> 6) * kWideTile + (row & 7) * 2;
#pragma unroll
        for (int e = 0; e < kTok; ++e)
          y[e] = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(col + tile_at<8>(kTok * quarter + e, (row & 63) >> 3)));
      }
      wait(&bars->p_done, par);
      tc_fence_after_sync();
      read16(trow + kTmP + kTok * quarter, x);
      wait(&bars->q_done, par);
      tc_fence_after_sync();
      {
        // dU0 = e^{G_63 - G} (K dS'^T) + M^T dO
        float m[kTok];
        read16(trow + kTmD + kTok * quarter, m);
#pragma unroll
        for (int e = 0; e < kTok; e += 4) {
          const float4 ge = gate[16 + e / 4];
          x[e] = ge.x * x[e] + m[e];
          x[e + 1] = ge.y * x[e + 1] + m[e + 1];
          x[e + 2] = ge.z * x[e + 2] + m[e + 2];
          x[e + 3] = ge.w * x[e + 3] + m[e + 3];
        }
      }
      put16<3>(trow + kTmX + kTok / 2 * quarter, 32, x);
      arrive(&bars->x_ready);
      // scale e^G dO takes the place of parts of dS' that are used up
      float eg[kTok];
#pragma unroll
      for (int e = 0; e < kTok; e += 4) {
        const float4 g = gate[e / 4];
        eg[e] = g.x;
        eg[e + 1] = g.y;
        eg[e + 2] = g.z;
        eg[e + 3] = g.w;
      }
#pragma unroll
      for (int e = 0; e < kTok; ++e) y[e] *= a.scale * eg[e];
      put16<3>(trow + kTmY + kTok / 2 * quarter, 32, y);
      arrive(&bars->u_ready);
      const float last = reinterpret_cast<const float*>(rest + W::kGate)[63];
      wait(&bars->e_done, par);
      tc_fence_after_sync();
      // dR; -e^G dX, dX = dV = b dR
      read16(trow + kTmP + kTok * quarter, x);
#pragma unroll
      for (int e = 0; e < kTok; e += 4) {
        const float4 be = gate[32 + e / 4];
        eg[e] *= -(be.x * x[e]);
        eg[e + 1] *= -(be.y * x[e + 1]);
        eg[e + 2] *= -(be.z * x[e + 2]);
        eg[e + 3] *= -(be.w * x[e + 3]);
      }
      put16<3>(trow + kTmW + kTok / 2 * quarter, 32, eg);
      arrive(&bars->w_ready);
      stage_parts(tiles + W::kM, row, 2 * quarter, x);
      unsigned char* col = rest + W::kV + kTok * quarter * 256 + row * 2;
#pragma unroll
      for (int e = 0; e < kTok; e += 4) {
        const float4 be = gate[32 + e / 4];
        const float bx[4] = {be.x * x[e], be.y * x[e + 1], be.z * x[e + 2], be.w * x[e + 3]};
#pragma unroll
        for (int f = 0; f < 4; ++f) *reinterpret_cast<__nv_bfloat16*>(col + (e + f) * 256) = __float2bfloat16_rn(bx[f]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->out_ready[st]);
      if (lane == 0) mbar_arrive(&bars->empty[st]);
      wait(&bars->d_done, par);
      tc_fence_after_sync();
#pragma unroll
      for (int i = 0; i < HS; i += 16) {
        float v[16], x2[16];
        read16(trow + kTmD + quarter * HS + i, v);
        read16(trow + kTmE + quarter * HS + i, x2);
#pragma unroll
        for (int e = 0; e < 16; ++e) S[i + e] = last * S[i + e] + (v[e] + x2[e]);
      }
    }
    if (active && a.dstate_in)
#pragma unroll
      for (int i = 0; i < HS; i += 4)
        *reinterpret_cast<float4*>(a.dstate_in + srow + i) = make_float4(S[i], S[i + 1], S[i + 2], S[i + 3]);
    tc_fence_before_sync();
  }
  settle(&bars->abort);
  __syncthreads();
  tc_fence_after_sync();
  if (warp == kTcWarps) tmem_dealloc(tm, 512);
}

template <typename K, typename A>
cudaError_t run_head(const LaunchEnv& env, K kernel, uint32_t smem, const A& a) {
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(unsigned(a.map.ndocs * a.Hv * ((a.dv + 127) / 128))), dim3(kTcThreads), smem,
                    env.stream, a);
}
template <int DK, HeadOut OUT>
cudaError_t run_head_walk(const LaunchEnv& env, const TcArgs& a) {
  return run_head(env, head_walk_kernel<DK, OUT>, TcShape<DK, OUT>::kSmem, a);
}

}  // namespace

cudaError_t launch_head_walk(const LaunchEnv& env, const DeltaArgs& f, const unsigned char* blocks,
                             const DeltaSave* save) {
  TcArgs a;
  a.q = f.q;
  a.k = f.k;
  a.v = f.v;
  a.Hk = f.Hk;
  a.Hv = f.Hv;
  a.dv = f.dv;
  a.T = f.T;
  a.map = f.map;
  a.scale = f.scale;
  a.state_in = f.state_in;
  a.state_out = f.state_out;
  a.out = f.out;
  a.out_fp32 = f.out_fp32;
  a.blocks = blocks;
  a.status = env.status;
  if (save) {
    a.save = *save;
    return f.dk == 64 ? run_head_walk<64, kSaved>(env, a) : run_head_walk<128, kSaved>(env, a);
  }
  if (f.out_fp32) return f.dk == 64 ? run_head_walk<64, kOutFp32>(env, a) : run_head_walk<128, kOutFp32>(env, a);
  return f.dk == 64 ? run_head_walk<64, kOutBf16>(env, a) : run_head_walk<128, kOutBf16>(env, a);
}

cudaError_t launch_head_reverse(const LaunchEnv& env, const ReverseArgs& r, int dk) {
  return dk == 64 ? run_head(env, head_reverse_kernel<64>, BackShape<64>::kSmem, r)
                  : run_head(env, head_reverse_kernel<128>, BackShape<128>::kSmem, r);
}

}  // namespace ittt
