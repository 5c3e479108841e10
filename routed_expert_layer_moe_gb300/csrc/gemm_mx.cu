// Steps 3 and 4 on MXFP4 experts: grouped per-expert products whose operands are E2M1 codes with
// one power-of-two scale per 32 values of the reduced dimension.
//
//   out[row][n] = sum over blocks k of 2^(sx[row][k] - 127) 2^(sw[n][k] - 127)
//                 sum_{i < 32} x[row][32 k + i] w[n][32 k + i]
//
// The tensor core applies both scales itself (tcgen05.mma kind::mxf4, scale factors in tensor
// memory) and sums the whole K range in fp32, so no partial sum ever leaves tensor memory: the
// FP8 / FP4 kernels with fp32 scales promote every 128-wide K block on the CUDA cores instead.
//
// Persistent CTAs, one per SM.  A unit is (slot, chunk of token rows, pair of weight tiles of 128
// or 64 rows, K split); gate/up: the pair is the gate and the up tile of the same columns.
// Token rows are the MMA's M side and the pair its N side, so a token's row lies in one thread of the
// epilogue: SwiGLU, the MXFP4 form of h (a block is 32 columns of the row) and the stores are
// row-local.  Two forms:
//   * One CTA: chunks of at most 128 rows, M = 128.  What decode needs: an expert's weights are
//     read once, and a chunk's token box is the smallest of 16 / 32 / 64 / 96 / 128 rows.
//   * SM pairs (PAIR; slots of 128 rows or more on average): clusters of two CTAs, chunks of at
//     most 256 rows, one cta_group::2 MMA with M = 256 over both CTAs' shared memory.  Each CTA stages
//     its half of the rows and one of the two weight tiles: 32 KB a stage, not 48, for the
//     same work of its tensor core.  What bounds large products is the way from L2 to shared memory:
//     without its MMAs and scales the one-CTA form took 0.50 us a stage of 48 KB (96 GB/s per SM),
//     against 0.27 us of MMAs.
// Roles of a CTA:
//   * Warp 0: TMA producer.  A stage is 256 codes (128 bytes) of K.
//   * Warp 1: issues a stage's four MMAs of K = 64.
//   * Warps 4-7: scales.  Per group of 512 codes (two stages) a thread copies the 16 scale bytes of
//     its row in each block of 128 rows (row-major in global memory) to shared memory, three
//     groups ahead; every warp then reads all rows and writes them to its lane quarter of tensor memory
//     in the order the MMA wants: for 128 rows and 128 codes, four columns, lane i of column q holding
//     the four bytes of row 32 q + i, the same in each quarter.  Copying them from shared memory
//     with tcgen05.cp instead put six copies a stage into the tensor core's queue: 0.69 us a stage,
//     0.62 without them.
//     A stage's scales are counted on the barrier of its copies and freed with them: with barriers
//     of their own, two more operations a group for the MMA warp, a dense gate/up product (8192 x 4096
//     by 28672 columns) took 391 us instead of 338.
//   * Warps 8-15: epilogue.  Columns 0-255 of tensor memory hold the unit's accumulators, the
//     columns above them the stages' scales.  The epilogue first moves the accumulators to
//     registers and hands them back, so only that move is not overlapped with the next unit's
//     MMAs; the copies run ahead through it.
//   * Every wait is bounded; on expiry the CTA drains its copies and MMAs, frees tensor memory,
//     reports MOE_FLAG_TIMEOUT and returns.
// Measured: decode reads its weights at 6.9 to 7.2 TB/s (128 tokens, 256 experts of 7168 x 2048: gate/up 563 us,
// down 295), 8192 tokens over 512 experts of 4096 x 1024 move 2.5 GB in 390 us and 1.85 GB in 273, and one
// expert of 4096 x 14336 takes 286 and 145 us: 6.7 PFLOP/s, where MMAs of K = 64 alone, back to back, take 220 and 110.
#include <algorithm>
#include <cmath>

#include "mx.cuh"

namespace moe {
namespace {

constexpr int STATS_CTAS = MOE_STATS_CTAS;
constexpr size_t STATS_BYTES = MOE_STATS_BYTES;
constexpr int BN = 128;                 // token rows of one CTA's chunk at most
constexpr int ROW_BYTES = 128;          // bytes of a row in one stage (one 128-byte swizzle span)
constexpr int KB = 256;                 // codes of a row in one stage
constexpr int TOK_BYTES = BN * ROW_BYTES;
constexpr int GROUP = 2;                // stages whose scales are loaded together (16 bytes of a row)
constexpr int SF_BUFS = 4;              // groups of scales in shared memory: three on their way while one is read
constexpr uint32_t SF_COL0 = 256;       // first tensor-memory column of the stages' scales
constexpr int MAX_STAGES = 6;           // their scales: 24 columns each at most
constexpr int NUM_THREADS = 512;        // four warpgroups
constexpr int SF_WARP0 = 4, SF_WARPS = 4;
constexpr int EPI_WARP0 = 8, EPI_WARPS = 8;
// Register split (setmaxnreg) of warpgroup 0, the scale warps and the two epilogue warpgroups (128
// accumulators a thread): what they add up to must be there at launch, which is checked before the first one.
// None of the forms spills with it; next to 220 KB of shared memory there is hardly an L1 to spill to.
constexpr int CTRL_REGS = 104, SF_REGS = 104, EPI_REGS = 152;
constexpr int SPLIT_REGS = 128 * (CTRL_REGS + SF_REGS + 2 * EPI_REGS);
constexpr uint32_t TMEM_COLS = 512;
constexpr long long TIMEOUT = 4000000000LL;  // SM cycles, about 2 s
// Token boxes of 16, 32, 64, 96 and 128 rows: the smallest that covers a chunk is copied.
constexpr int NUM_BOXES = 5;
__host__ __device__ constexpr int box_rows(int i) { return i ? 32 * i : 16; }
__host__ __device__ constexpr int box_of(int rows) { return rows <= 16 ? 0 : (rows + 31) / 32; }

// Sizes that go with TW, the rows of one weight tile (64 or 128), and the form.
template <int TW, bool PAIR>
struct Tile {
  static constexpr int W_BYTES = TW * ROW_BYTES;
  static constexpr int W_STAGED = PAIR ? W_BYTES : 2 * W_BYTES;  // weight bytes of this CTA's stage
  static constexpr int STAGE = W_STAGED + TOK_BYTES;             // weights | tokens
  static constexpr int NB = 2 * TW / 128;                        // 128-row scale blocks of a pair's rows
  static constexpr int SF_BUF = (1 + NB) * 128 * 16;             // one group's scales in shared memory
  static constexpr int SF_COLS = 2 * (4 * NB + 4);               // one stage's in tensor memory: weights, then tokens
};

struct MxParams {
  int mode;          // MODE_SWIGLU or MODE_DOWN
  int nslots, masked, M_max;
  int K;             // codes of a row
  int kb_total;      // stages of the K range
  int kb_per_split;  // stages of a split: even, so that groups start on 16 scale bytes
  int ksplit;
  int NA;            // weight rows per slot
  int pairs;         // tile pairs per token chunk
  int pair_stride;   // weight rows between pairs
  int a1_off;        // row of the pair's second tile relative to the first
  int out_cols;
  int stages;
  int boxes;           // token boxes with a tensor map: enough for any chunk
  int early;           // the kernel before this one is the gate/up GEMM of the same call
  int vec_tok, vec_w;  // scale rows may be read 16 bytes at a time
  const uint8_t* w_scales;    // [slots * NA][K/32]
  const uint8_t* act_scales;  // [rows][K/32]
  const int32_t* masked_m;
  const int32_t* offsets;
  void* out;            // gate/up: MXFP4 codes [rows][out_cols/2]; down: bf16 [rows][out_cols]
  uint8_t* out_scales;  // gate/up: [rows][out_cols/32]
  float* part;          // split K: [ksplit][rows_total][out_cols]
  long rows_total;
  int32_t* err;
  int* stats;
  uint32_t sf_off, pre_off, bar_off, misc_off;
};

struct TokenMaps {
  CUtensorMap box[NUM_BOXES];
};

struct Unit {
  int s, c, j, q;
  int nvalid;        // token rows of this CTA's chunk
  int most;          // the larger of a pair's two chunks (one CTA: nvalid)
  int rowB;          // first grouped-buffer row of this CTA's chunk
  int rowA0, rowA1;  // first weight row of each tile
  int kb0, kb1;      // stages
  bool a1;           // the second tile exists
};

template <bool PAIR, bool SPLIT>
__device__ __forceinline__ Unit decode_unit(const MxParams& p, const int* prefix, const int* srows, const int* sbase,
                                            int u, uint32_t rank) {
  constexpr int CH = PAIR ? 2 * BN : BN;
  int lo = 0, hi = p.nslots;  // prefix[lo] <= u < prefix[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= u)
      lo = mid;
    else
      hi = mid;
  }
  Unit U;
  U.s = lo;
  const int r = u - prefix[lo];
  const int m = srows[lo];
  const int nch = (m + CH - 1) / CH;
  U.q = SPLIT ? r % p.ksplit : 0;
  const int rest = SPLIT ? r / p.ksplit : r;
  U.c = rest % nch;
  U.j = rest / nch;
  const int base = m / nch, extra = m - base * nch;  // near-equal chunks
  U.nvalid = base + (U.c < extra ? 1 : 0);
  U.rowB = sbase[lo] + U.c * base + min(U.c, extra);
  U.most = U.nvalid;
  if constexpr (PAIR) {  // rank 0 takes the first half of the rows (rounded up)
    const int n0 = (U.nvalid + 1) >> 1;
    U.most = n0;
    if (rank) {
      U.rowB += n0;
      U.nvalid -= n0;
    } else {
      U.nvalid = n0;
    }
  }
  U.rowA0 = lo * p.NA + U.j * p.pair_stride;
  U.rowA1 = U.rowA0 + p.a1_off;
  U.a1 = PAIR || p.mode == MODE_SWIGLU || U.j * p.pair_stride + p.a1_off < p.NA;
  U.kb0 = SPLIT ? U.q * p.kb_per_split : 0;
  U.kb1 = SPLIT ? min(p.kb_total, U.kb0 + p.kb_per_split) : p.kb_total;
  return U;
}

__device__ __forceinline__ uint64_t policy_evict_normal() {
  uint64_t pol;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol));
  return pol;
}

// One lane of a converged warp, the same at every call.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n"
      "  .reg .pred p;\n"
      "  elect.sync _|p, 0xffffffff;\n"
      "  selp.u32 %0, 1, 0, p;\n"
      "}\n"
      : "=r"(one));
  return one;
}

// D[tmem] (+)= (A sfa) (B sfb)^T over K = 64 codes, issued by one thread.  PAIR: by the leader for both
// CTAs; D, sfa and sfb are at the same addresses of both tensor memories.
template <bool PAIR>
__device__ __forceinline__ void mma_mxf4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                         uint32_t sfb, uint32_t accumulate) {
  if constexpr (PAIR)
    asm volatile(
        "{\n"
        "  .reg .pred p;\n"
        "  setp.ne.b32 p, %6, 0;\n"
        "  tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n"
        "}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n"
        "  .reg .pred p;\n"
        "  setp.ne.b32 p, %6, 0;\n"
        "  tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n"
        "}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

// Instruction descriptor of kind::mxf4: E2M1 x E2M1 with UE8M0 scales, K-major; the scale factor
// id (0 or 2) picks the two bytes of a scale word that a K = 64 step uses.
__device__ __forceinline__ uint32_t mx_idesc(int M, int N, uint32_t sf_id) {
  return (sf_id << 4)                  // B scale factor id
         | (1u << 7)                   // A: E2M1
         | (1u << 10)                  // B: E2M1
         | ((uint32_t)(N >> 3) << 17)  // N / 8
         | (1u << 23)                  // scales: UE8M0
         | ((uint32_t)(M >> 4) << 24)  // M / 16
         | (sf_id << 29);              // A scale factor id
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void cp_async4_at(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// N (32 or 64) columns of this thread's lane of tensor memory, not waited for.
template <int N>
__device__ __forceinline__ void tmem_load(uint32_t taddr, float (&v)[N]) {
#pragma unroll
  for (int o = 0; o < N; o += 32)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
                 : "=f"(v[o + 0]), "=f"(v[o + 1]), "=f"(v[o + 2]), "=f"(v[o + 3]), "=f"(v[o + 4]), "=f"(v[o + 5]), "=f"(v[o + 6]), "=f"(v[o + 7]), "=f"(v[o + 8]), "=f"(v[o + 9]), "=f"(v[o + 10]), "=f"(v[o + 11]), "=f"(v[o + 12]), "=f"(v[o + 13]), "=f"(v[o + 14]), "=f"(v[o + 15]),
                   "=f"(v[o + 16]), "=f"(v[o + 17]), "=f"(v[o + 18]), "=f"(v[o + 19]), "=f"(v[o + 20]), "=f"(v[o + 21]), "=f"(v[o + 22]), "=f"(v[o + 23]), "=f"(v[o + 24]), "=f"(v[o + 25]), "=f"(v[o + 26]), "=f"(v[o + 27]), "=f"(v[o + 28]), "=f"(v[o + 29]), "=f"(v[o + 30]), "=f"(v[o + 31])
                 : "r"(taddr + (uint32_t)o)
                 : "memory");
}

// Wait for this thread's loads; v is what one of them wrote.
template <int N>
__device__ __forceinline__ void tmem_loaded(float (&v)[N]) {
#pragma unroll
  for (int o = 0; o < N; o += 32)
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[o + 0]), "+f"(v[o + 1]), "+f"(v[o + 2]), "+f"(v[o + 3]), "+f"(v[o + 4]), "+f"(v[o + 5]), "+f"(v[o + 6]), "+f"(v[o + 7]), "+f"(v[o + 8]), "+f"(v[o + 9]), "+f"(v[o + 10]), "+f"(v[o + 11]), "+f"(v[o + 12]), "+f"(v[o + 13]), "+f"(v[o + 14]), "+f"(v[o + 15]),
                   "+f"(v[o + 16]), "+f"(v[o + 17]), "+f"(v[o + 18]), "+f"(v[o + 19]), "+f"(v[o + 20]), "+f"(v[o + 21]), "+f"(v[o + 22]), "+f"(v[o + 23]), "+f"(v[o + 24]), "+f"(v[o + 25]), "+f"(v[o + 26]), "+f"(v[o + 27]), "+f"(v[o + 28]), "+f"(v[o + 29]), "+f"(v[o + 30]), "+f"(v[o + 31])
                 :
                 : "memory");
}

// Four columns of this warp's 32 lanes of tensor memory.
__device__ __forceinline__ void tmem_st4(uint32_t taddr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}

__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// h = SiLU(g) u of a pair, with the special-function unit's exponential and reciprocal (2 ulp and 1 ulp): for
// g -> -inf the exponential is inf and the product -0 u.  h is rounded to four bits next; a value within those ulps of
// a tie may take the neighbouring code, as it may after another order of the fp32 sum behind g and u.  Against 64
// bits one expert of 14336 is as far off as a plain form with expf and an IEEE division (1.68e-3 both; 8e-5 between
// the two).
__device__ __forceinline__ float2 silu_mul(float2 g, float2 u) {
  const float2 t = __fmul2_rn(g, make_float2(-1.4426950408889634f, -1.4426950408889634f));
  float2 e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
  e = __fadd2_rn(e, make_float2(1.0f, 1.0f));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(e.x));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(e.y));
  return __fmul2_rn(__fmul2_rn(g, e), u);
}

// Units of 32 bytes, four a lane, exchanged within each four lanes: unit u of lane l becomes unit l of
// lane u.  A store then writes 128 bytes of one row from four neighbours instead of 32 bytes of
// each of 32 rows, which took 45 cycles.
__device__ __forceinline__ void quad_transpose(uint32_t (&w)[4][8], int lane) {
#pragma unroll
  for (int step = 1; step <= 2; step <<= 1) {
    const bool up = lane & step;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (u & step) continue;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? w[u][i] : w[u + step][i], step);
        if (up)
          w[u][i] = got;
        else
          w[u + step][i] = got;
      }
    }
  }
}

// The four units of every lane to rows base + u (u = 0..3) of out, base the lane's row rounded down to
// a multiple of four; `rows` of them exist.  dst(row) is where the units of a row begin.
template <typename F>
__device__ __forceinline__ void store_quad(uint32_t (&w)[4][8], int lane, int base, int rows, bool wide, F dst) {
  quad_transpose(w, lane);
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    if (base + u < rows) {
      uint8_t* d = dst(base + u) + 32 * (lane & 3);
      const uint4 a = make_uint4(w[u][0], w[u][1], w[u][2], w[u][3]), b = make_uint4(w[u][4], w[u][5], w[u][6], w[u][7]);
      if (wide) {
        st_global_v8(d, a, b);
      } else {
        reinterpret_cast<uint4*>(d)[0] = a;
        reinterpret_cast<uint4*>(d)[1] = b;
      }
    }
  }
}

// SPLIT: the K range is split (down only); partial sums go to the workspace.
template <int MODE, int TW, bool PAIR, bool SPLIT>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    grouped_gemm_mx_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ TokenMaps tmB,
                           const MxParams p) {
  using L = Tile<TW, PAIR>;
  constexpr int TC = TW / 2;  // columns of each tile that an epilogue thread holds
  constexpr int CH = PAIR ? 2 * BN : BN;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);  // pointer arithmetic: it stays in the shared space
  uint8_t* sf = smem + p.sf_off;                           // [SF_BUFS][1 + NB blocks][128 rows][16]
  int* prefix = reinterpret_cast<int*>(smem + p.pre_off);  // [nslots + 1] unit prefix
  int* srows = prefix + p.nslots + 1;                      // [nslots] valid rows per slot
  int* sbase = srows + p.nslots;                           // [nslots] first grouped-buffer row per slot
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + p.bar_off);
  uint64_t* empty = full + p.stages;
  uint64_t* tfull = empty + p.stages;    // accumulators written
  uint64_t* tempty = tfull + 1;          // accumulators read
  uint64_t* drain = tempty + 1;
  uint64_t* fin = drain + 1;             // pairs: the peer CTA is done with this CTA's memory
  uint32_t* tmem_base_smem = reinterpret_cast<uint32_t*>(smem + p.misc_off);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + p.misc_off + 4);

  const int tid = threadIdx.x;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;  // the warp number is uniform
  // pairs: rank 0 (the leader) issues the MMAs; units are dealt per cluster
  const uint32_t crank = PAIR ? cluster_ctarank() : 0u;
  const bool leader = crank == 0;
  const int unit0 = PAIR ? (int)cluster_id_x() : (int)blockIdx.x;
  const int ustride = PAIR ? (int)nclusters_x() : (int)gridDim.x;

  if (tid == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&full[i], 1 + (PAIR ? 2 * SF_WARPS : SF_WARPS));  // the copies, and the scale warps
      mbar_init(&empty[i], 1);
    }
    mbar_init(tfull, 1);
    mbar_init(tempty, PAIR ? 2 * EPI_WARPS : EPI_WARPS);
    mbar_init(drain, 1);
    mbar_init(fin, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc<PAIR>(tmem_base_smem, TMEM_COLS);
    tmem_relinquish<PAIR>();
  }
  // Launched while the kernel before it in the stream still runs.  If that one is the gate/up GEMM
  // of the same call, everything before it has finished (its CTAs wait here, then let this kernel
  // start), the row counts and the weights among it: only h has to be waited for, below.
  if (!p.early) grid_dependency_wait();
  grid_dependents_launch();
  for (int s = tid; s < p.nslots; s += NUM_THREADS) {
    int m = __ldcg(p.masked_m + s);  // not through the read-only path: written while this kernel may have begun
    if (p.masked) m = min(m, p.M_max);
    m = max(m, 0);
    srows[s] = m;
    sbase[s] = p.masked ? s * p.M_max : __ldcg(p.offsets + s);
    prefix[s + 1] = (m + CH - 1) / CH * p.pairs * p.ksplit;
  }
  if (tid == 0) prefix[0] = 0;
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 0) {
    int run = 0;
    for (int base = 1; base <= p.nslots; base += 32) {
      const int i = base + lane;
      int v = (i <= p.nslots) ? prefix[i] : 0;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int n = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v += n;
      }
      if (i <= p.nslots) prefix[i] = run + v;
      run += __shfl_sync(0xffffffffu, v, 31);
    }
  }
  __syncthreads();
  // both CTAs' barriers are initialised before either CTA touches the other's
  if constexpr (PAIR) cluster_sync_all();
  tc_fence_after_sync();
  const uint32_t tmem_base = __shfl_sync(0xffffffffu, *tmem_base_smem, 0);  // uniform, as the tensor core's operands are
  const int total = prefix[p.nslots];
  auto unit = [&](int u) { return decode_unit<PAIR, SPLIT>(p, prefix, srows, sbase, u, crank); };

  if (warp < SF_WARP0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(CTRL_REGS));
    if (warp == 0) {
      // ------------------------------------------------------------ producer
      if (lane == 0) {
        tma_prefetch_map(&tmA);
        for (int i = 0; i < p.boxes; ++i) tma_prefetch_map(&tmB.box[i]);
        // Weights give way in L2 to what is used again, but not in the down product of SM pairs: with 512 experts of
        // 1024 x 4096 it took 319 us so and 267 without (one expert of 14336 x 4096: 145 and 147).
        const uint64_t pol = PAIR && MODE == MODE_DOWN ? policy_evict_normal() : policy_evict_first();
        int stage = 0;
        uint32_t phase = 0;
        long issued = 0;
        bool ok = true;
        auto box = [&](const Unit& U) { return min(box_of(U.most), p.boxes - 1); };
        // a stage's byte count and its weights; pairs: the leader's barrier counts both CTAs' copies
        auto load_weights = [&](const Unit& U, int kb, int at) {
          uint8_t* st = smem + (size_t)at * L::STAGE;
          const int x = kb * ROW_BYTES;
          const uint32_t tok = (uint32_t)box_rows(box(U)) * ROW_BYTES;
          if constexpr (PAIR) {
            if (leader) {
              mbar_arrive_expect_tx(&full[at], 2u * (L::W_BYTES + tok));
              tma_load_2d_hint(st, &tmA, &full[at], x, U.rowA0, pol);
            } else {
              tma_load_2d_pair_hint(st, &tmA, mapa_shared(&full[at], 0), x, U.rowA1, pol);
            }
          } else {
            mbar_arrive_expect_tx(&full[at], (U.a1 ? 2u : 1u) * L::W_BYTES + tok);
            tma_load_2d_hint(st, &tmA, &full[at], x, U.rowA0, pol);
            if (U.a1) tma_load_2d_hint(st + L::W_BYTES, &tmA, &full[at], x, U.rowA1, pol);
          }
        };
        int ahead = 0;  // stages of the first unit whose weights are on their way before h may be read
        if (p.early) {
          if (unit0 < total) {
            const Unit U = unit(unit0);
            for (ahead = 0; ahead < p.stages && U.kb0 + ahead < U.kb1; ++ahead) load_weights(U, U.kb0 + ahead, ahead);
          }
          grid_dependency_wait();
        }
        for (int u = unit0; ok && u < total; u += ustride) {
          const Unit U = unit(u);
          const CUtensorMap* mb = &tmB.box[box(U)];
          for (int kb = U.kb0; kb < U.kb1; ++kb) {
            if (ahead > 0) {
              --ahead;
            } else {
              if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, TIMEOUT)) {
                ok = false;
                break;
              }
              load_weights(U, kb, stage);
            }
            uint8_t* st = smem + (size_t)stage * L::STAGE;
            const int x = kb * ROW_BYTES;
            if (PAIR && !leader)
              tma_load_2d_pair(st + L::W_STAGED, mb, mapa_shared(&full[stage], 0), x, U.rowB);
            else
              tma_load_2d(st + L::W_STAGED, mb, &full[stage], x, U.rowB);
            ++issued;
            if (++stage == p.stages) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
        if (!ok && issued > 0) {
          // let the copies already in flight land before the CTA's shared memory is released
          const uint64_t t0 = global_timer_ns();
          while (global_timer_ns() - t0 < 200000u) {
          }
        }
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMAs
      // The whole warp runs the loop and one elected lane issues: the operands then stay in uniform
      // registers.  In a loop that only lane 0 ran, each MMA took its eight operands there one by one, 85
      // cycles an MMA and 680 a stage of 528 cycles of MMAs.
      auto commit = [&](uint64_t* bar) {
        if constexpr (PAIR)
          tc_commit_pair(bar, 3);  // both CTAs' barriers
        else
          tc_commit(bar);
      };
      const uint64_t desc_w = smem_desc_sw128(smem_u32(smem)), desc_t = smem_desc_sw128(smem_u32(smem) + L::W_STAGED);
      int stage = 0;
      uint32_t phase = 0, u_it = 0;
      bool ok = true, any = false;
      // whole K and always two weight tiles: a unit need not be looked up between its MMAs and the next's
      constexpr bool ALIKE = MODE == MODE_SWIGLU;
      int kb0 = 0, kb1 = p.kb_total, N = 2 * TW;
      for (int u = unit0; ok && leader && u < total; u += ustride, ++u_it) {
        if constexpr (!ALIKE) {
          const Unit U = unit(u);
          kb0 = __shfl_sync(0xffffffffu, U.kb0, 0), kb1 = __shfl_sync(0xffffffffu, U.kb1, 0);
          N = __shfl_sync(0xffffffffu, U.a1 ? 2 * TW : TW, 0);
        }
        const uint32_t id0 = mx_idesc(PAIR ? 2 * BN : BN, N, 0), id2 = mx_idesc(PAIR ? 2 * BN : BN, N, 2);
        ok = __all_sync(0xffffffffu, mbar_wait(tempty, (u_it & 1u) ^ 1u, abort_flag, TIMEOUT));
        if (!ok) break;
        tc_fence_after_sync();
        for (int kb = kb0; kb < kb1; ++kb) {
          ok = __all_sync(0xffffffffu, mbar_wait(&full[stage], phase, abort_flag, TIMEOUT));
          if (!ok) break;
          tc_fence_after_sync();
          const uint64_t dw = desc_w + (uint32_t)stage * (L::STAGE >> 4), dtok = desc_t + (uint32_t)stage * (L::STAGE >> 4);
          const uint32_t scol = tmem_base + SF_COL0 + (uint32_t)stage * L::SF_COLS;
          const bool both = p.K - kb * KB > KB / 2;  // a last stage may be half a stage
          if (elect_one()) {
#pragma unroll
            for (uint32_t j = 0; j < 2; ++j) {
              if (j == 0 || both) {
                const uint32_t sfb = scol + 4 * L::NB * j, sfa = scol + 8 * L::NB + 4 * j;
                mma_mxf4<PAIR>(tmem_base, dtok + 4 * j, dw + 4 * j, id0, sfa, sfb, kb > kb0 || j > 0);
                mma_mxf4<PAIR>(tmem_base, dtok + 4 * j + 2, dw + 4 * j + 2, id2, sfa, sfb, 1u);
              }
            }
            commit(&empty[stage]);
          }
          __syncwarp();
          any = true;
          if (++stage == p.stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (ok && elect_one()) commit(tfull);
        __syncwarp();
      }
      if (!ok && any && elect_one()) {
        // all MMAs issued by this thread must finish before tensor memory is freed
        if constexpr (PAIR)
          tc_commit_pair(drain, 1);
        else
          tc_commit(drain);
        const long long t0 = clock64();
        while (!mbar_try_wait(drain, 0) && clock64() - t0 < TIMEOUT) {
        }
      }
      __syncwarp();
    } else if (warp == 2) {
      // ------------------------------------------------------------ statistics
      if (lane == 0 && p.stats) {
        int units = 0, tiles = 0;
        for (int u = unit0; leader && u < total; u += ustride) {
          const Unit U = unit(u);
          ++units;
          tiles += (U.j == 0 && U.q == 0);  // one unit per (slot, token chunk)
        }
        if (p.early) grid_dependency_wait();  // the kernel ahead writes the same counters
        for (int h = 0; h < 2; ++h) {
          if (blockIdx.x < STATS_CTAS) {
            p.stats[(h * STATS_CTAS + blockIdx.x) * 2] = h ? 0 : units;
            p.stats[(h * STATS_CTAS + blockIdx.x) * 2 + 1] = h ? 0 : tiles;
          }
          if (blockIdx.x == 0)
            for (int c = gridDim.x; c < STATS_CTAS; ++c) {
              p.stats[(h * STATS_CTAS + c) * 2] = 0;
              p.stats[(h * STATS_CTAS + c) * 2 + 1] = 0;
            }
        }
      }
    }
  } else if (warp < EPI_WARP0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(SF_REGS));
    // ------------------------------------------------------------ scales
    // These warps run a serial chain per group, and it bounds large products: 1200-1400 cycles a turn
    // against 1056 of the group's MMAs.  So addresses are per unit, all reads of a turn come before its
    // stores, the next copies are requested while those are on their way, and the next unit is
    // looked up after the MMA thread has been told (dense gate/up 294 -> 286 us).
    const int lt = tid - SF_WARP0 * 32;  // this thread's row of each 128-row block
    const uint32_t words = (uint32_t)p.K / 128;  // words of a scale row
    const size_t row_bytes = (size_t)p.K / 32;
    const uint32_t t_lane = tmem_base + ((uint32_t)((warp & 3) * 32) << 16) + SF_COL0;
    // The groups of all units in order, requested SF_BUFS - 1 groups ahead.  Rows past the chunk, a
    // missing second tile and codes past K keep what shared memory holds: no MMA result that is
    // used depends on them.
    int u = unit0, left = 0;  // the next group to request: its unit and the unit's stages that are left
    const uint8_t *pt = nullptr, *pw[L::NB];
    uint32_t w0 = 0;  // its first word of a scale row
    int requested = 0;
    uint32_t single = 0;  // bit r % 32: group r, at the end of its unit, has one stage
    auto next_unit = [&]() {
      if (u >= total) return;
      const Unit U = unit(u);
      left = U.kb1 - U.kb0;
      w0 = (uint32_t)U.kb0 * 2;
      pt = lt < U.nvalid ? p.act_scales + (size_t)(U.rowB + lt) * row_bytes + 4 * w0 : nullptr;
#pragma unroll
      for (int i = 0; i < L::NB; ++i) {
        const int r = 128 * i + lt;
        const int row = r >= TW ? U.rowA1 + r - TW : U.rowA0 + r;
        pw[i] = r < TW || U.a1 ? p.w_scales + (size_t)row * row_bytes + 4 * w0 : nullptr;
      }
    };
    // The 16 scale bytes of a row's codes from word w0 on, those that exist.
    auto fetch = [&](uint32_t dst, const uint8_t* src, bool vec) {
      if (vec) {
        cp_async16(dst, src);
      } else {
        for (uint32_t i = 0; i < 4 && w0 + i < words; ++i) cp_async4_at(dst + 4 * i, src + 4 * i);
      }
    };
    const uint32_t sf0 = smem_u32(sf) + (uint32_t)lt * 16;
    auto request = [&](uint32_t buf) {
      if (u < total) {
        const uint32_t dst = sf0 + buf * L::SF_BUF;
        if (pt) {
          fetch(dst, pt, p.vec_tok);
          pt += 16;
        }
#pragma unroll
        for (int i = 0; i < L::NB; ++i) {
          if (pw[i]) {
            fetch(dst + 2048u * (1 + i), pw[i], p.vec_w);
            pw[i] += 16;
          }
        }
        const uint32_t bit = 1u << (requested & 31);
        single = left == 1 ? single | bit : single & ~bit;
        ++requested;
        w0 += 4;
        left -= GROUP;
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto look_up = [&]() {  // the unit of the next request
      if (left <= 0 && u < total) {
        u += ustride;
        next_unit();
      }
    };
    next_unit();
    if (p.early) grid_dependency_wait();  // for the scales of h
    for (uint32_t i = 0; i < SF_BUFS - 1; ++i) {
      request(i);
      look_up();
    }
    // The stores of a turn are done: tell the MMA thread, through the barrier of the stage that also
    // counts its copies (the leader's, for both CTAs of a pair).
    auto arrive = [&](uint64_t* bar) {
      if (PAIR)
        mbar_arrive_remote(mapa_shared(bar, 0));
      else
        mbar_arrive(bar);
    };
    auto release = [&](int stage, bool two) {
      asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        arrive(&full[stage]);
        if (two) arrive(&full[stage + 1 == p.stages ? 0 : stage + 1]);
      }
    };
    uint32_t buf = 0, phase = 0;
    int stage = 0;
    bool ok = true;
    for (int turn = 0; turn < requested; ++turn) {
      asm volatile("cp.async.wait_group %0;" ::"n"(SF_BUFS - 2) : "memory");  // this turn's group is here
      // The four warps' rows of the group, and the end of their reads of the buffer before it.  Every
      // warp takes every turn, after a wait that gave up too, so this barrier always completes.
      asm volatile("bar.sync 1, 128;" ::: "memory");
      const bool two = !(single >> (turn & 31) & 1u);
      const uint4* src = reinterpret_cast<const uint4*>(sf + buf * L::SF_BUF) + lane;
      const uint32_t nb = buf == 0 ? SF_BUFS - 1 : buf - 1;
      if (++buf == SF_BUFS) buf = 0;
      uint4 v[1 + L::NB][4];  // all of the group's reads before its first store
#pragma unroll
      for (int b = 0; b <= L::NB; ++b)
#pragma unroll
        for (int q = 0; q < 4; ++q) v[b][q] = src[128 * b + 32 * q];
      // the group's last stage is free, and with it the one before; the whole warp goes on or gives
      // up: its stores to tensor memory are warp-wide
      const bool wraps = stage + 1 == p.stages;
      const int s1 = wraps ? 0 : stage + 1;
      const int end = two ? s1 : stage;
      const uint32_t ephase = two && wraps ? phase ^ 1u : phase;
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&empty[end], ephase ^ 1u, abort_flag, TIMEOUT));
      if (!ok) {
        request(nb);
        look_up();
        continue;
      }
      tc_fence_after_sync();
      const uint32_t c0 = t_lane + (uint32_t)stage * L::SF_COLS, c1 = t_lane + (uint32_t)s1 * L::SF_COLS;
      auto at = [](int b) { return (uint32_t)(b == 0 ? 8 * L::NB : 4 * (b - 1)); };  // tokens, then the weights' blocks
      auto step = [](int b) { return (uint32_t)(b == 0 ? 4 : 4 * L::NB); };
#pragma unroll
      for (int b = 0; b <= L::NB; ++b) {
        tmem_st4(c0 + at(b), v[b][0].x, v[b][1].x, v[b][2].x, v[b][3].x);
        tmem_st4(c0 + at(b) + step(b), v[b][0].y, v[b][1].y, v[b][2].y, v[b][3].y);
      }
      if (two) {
#pragma unroll
        for (int b = 0; b <= L::NB; ++b) {
          tmem_st4(c1 + at(b), v[b][0].z, v[b][1].z, v[b][2].z, v[b][3].z);
          tmem_st4(c1 + at(b) + step(b), v[b][0].w, v[b][1].w, v[b][2].w, v[b][3].w);
        }
      }
      request(nb);  // while the stores are on their way
      release(stage, two);
      look_up();  // a few hundred cycles: after the group that the MMA thread waits for
      const int next = two ? s1 + 1 : stage + 1;  // the stage after the group's last
      if (two && wraps) phase ^= 1u;
      stage = next;
      if (stage == p.stages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    cp_async_wait_all();  // no copy may land after the CTA has exited
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(EPI_REGS));
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3;              // tensor-memory lane quarter this warp may access
    const int half = (warp - EPI_WARP0) >> 2;  // column half of each tile
    const int lrow = quarter * 32 + lane;      // token row of this thread
    const uint32_t t_lane = tmem_base + ((uint32_t)(quarter * 32) << 16);
    const int c_lo = half * TC;
    const size_t oc = (size_t)p.out_cols;
    uint32_t u_it = 0;
    for (int u = unit0; u < total; u += ustride, ++u_it) {
      const Unit U = unit(u);
      // the whole warp goes on together (its tensor-memory loads are warp-wide) or gives up together
      if (!__all_sync(0xffffffffu, mbar_wait(tfull, u_it & 1u, abort_flag, TIMEOUT))) break;
      tc_fence_after_sync();
      const bool warp_live = quarter * 32 < U.nvalid;
      const bool live = lrow < U.nvalid;
      // once per unit: the accumulators are in registers
      auto release = [&]() {
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          if (PAIR)
            mbar_arrive_remote(mapa_shared(tempty, 0));
          else
            mbar_arrive(tempty);
        }
      };
      if (!warp_live) {  // rows past the chunk: nothing to read or store
        release();
        continue;
      }
      const uint32_t t0 = t_lane + (uint32_t)c_lo;
      if constexpr (MODE == MODE_SWIGLU) {
        float acc0[TC], acc1[TC];
        tmem_load<TC>(t0, acc0);
        tmem_load<TC>(t0 + (uint32_t)TW, acc1);
        tmem_loaded<TC>(acc0);
        tmem_loaded<TC>(acc1);
        release();
#pragma unroll
        for (int i = 0; i < TC; i += 2) {
          const float2 h = silu_mul(make_float2(acc0[i], acc0[i + 1]), make_float2(acc1[i], acc1[i + 1]));
          acc0[i] = h.x, acc0[i + 1] = h.y;
        }
        uint32_t code[TC / 8], sb[TC / 32];
#pragma unroll
        for (int b = 0; b < TC / 32; ++b) {
          float amax = 0.0f;
#pragma unroll
          for (int i = 0; i < 32; i += 2) amax = mx_amax3(amax, acc0[32 * b + i], acc0[32 * b + i + 1]);
          sb[b] = mx_scale_byte(amax);
          const float inv = mx_inv_scale(sb[b]);
#pragma unroll
          for (int i = 0; i < 4; ++i) code[4 * b + i] = mx_codes8(acc0 + 32 * b + 8 * i, inv);
        }
        if (!live) continue;
        const size_t row = (size_t)(U.rowB + lrow);
        const size_t col = (size_t)U.j * TW + c_lo;
        uint8_t* dst = static_cast<uint8_t*>(p.out) + row * (oc / 2) + col / 2;
        uint8_t* ds = p.out_scales + row * (oc / 32) + col / 32;
        if constexpr (TC == 64) {
          const uint4 a = make_uint4(code[0], code[1], code[2], code[3]), b = make_uint4(code[4], code[5], code[6], code[7]);
          if ((reinterpret_cast<uintptr_t>(p.out) & 31u) == 0) {
            st_global_v8(dst, a, b);
          } else {
            reinterpret_cast<uint4*>(dst)[0] = a;
            reinterpret_cast<uint4*>(dst)[1] = b;
          }
          *reinterpret_cast<uint16_t*>(ds) = (uint16_t)(sb[0] | (sb[1] << 8));
        } else {
          *reinterpret_cast<uint4*>(dst) = make_uint4(code[0], code[1], code[2], code[3]);
          *ds = (uint8_t)sb[0];
        }
      } else {
        static_assert(MODE == MODE_SWIGLU || TC == 64, "64 columns of each tile a thread");
        const size_t col = (size_t)U.j * p.pair_stride + c_lo;
        const int base = lrow & ~3;
        if constexpr (SPLIT) {
          float acc0[64], acc1[64];
          tmem_load<64>(t0, acc0);
          tmem_load<64>(t0 + (uint32_t)TW, acc1);
          tmem_loaded<64>(acc0);
          tmem_loaded<64>(acc1);
          release();
          float* part = p.part + ((size_t)U.q * p.rows_total + U.rowB) * oc + col;
          const bool wide = (reinterpret_cast<uintptr_t>(p.part) & 31u) == 0;
          auto store = [&](const float* a, int c) {  // 32 columns from column c on
            uint32_t w[4][8];
#pragma unroll
            for (int i = 0; i < 32; ++i) w[i / 8][i % 8] = __float_as_uint(a[i]);
            store_quad(w, lane, base, U.nvalid, wide,
                       [&](int r) { return reinterpret_cast<uint8_t*>(part + (size_t)r * oc + c); });
          };
          store(acc0, 0);
          store(acc0 + 32, 32);
          if (U.a1) {
            store(acc1, TW);
            store(acc1 + 32, TW + 32);
          }
        } else {
          // a tile is packed to bf16 before the next one is loaded: with both in registers the compiler
          // spilled (dense down product 203 us, not 172)
          uint32_t w[2][4][8];
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            float a[64];
            tmem_load<64>(t0 + (uint32_t)(t * TW), a);
            tmem_loaded<64>(a);
#pragma unroll
            for (int i = 0; i < 32; ++i) w[t][i / 8][i % 8] = bf16x2(a[2 * i], a[2 * i + 1]);
          }
          release();
          __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + (size_t)U.rowB * oc + col;
          const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (t == 0 || U.a1)
              store_quad(w[t], lane, base, U.nvalid, wide,
                         [&](int r) { return reinterpret_cast<uint8_t*>(out + (size_t)r * oc + t * TW); });
          }
        }
      }
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if constexpr (PAIR) {
    // Neither CTA frees its tensor memory or leaves while the other may still use it: the leader's
    // MMAs read the peer's shared memory and write its tensor memory, the peer's copies and
    // arrivals land on the leader's barriers.  Each tells the other that it is done and waits,
    // bounded, for the other's word.
    if (tid == 0) {
      mbar_arrive_remote(mapa_shared(fin, crank ^ 1u));
      const long long t0 = clock64();
      while (!mbar_try_wait<true>(fin, 0)) {
        if (clock64() - t0 > TIMEOUT) {
          *abort_flag = 1;
          break;
        }
      }
    }
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc<PAIR>(tmem_base, TMEM_COLS);
  }
  if (tid == 0 && *abort_flag) atomicOr(p.err, MOE_FLAG_TIMEOUT);
  if (p.early) grid_dependency_wait();  // a CTA without units: this kernel never ends before the one ahead
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

// SM pairs for slots of prefill size: 128 rows or more on average.  The down product needs whole
// pairs of weight tiles (H a multiple of 256).
bool use_pairs(const moe_problem& p, int mode) {
  return (double)p.T * p.K / std::max(1, p.P) >= 128.0 && (mode == MODE_SWIGLU || p.H % 256 == 0);
}

struct Plan {
  bool pair;
  int tw, kb_total, kb_per_split, ksplit, pairs, stages;
  size_t smem, part_bytes;
  uint32_t sf_off, pre_off, bar_off, misc_off;
};

// Share of the SMs' time that `units` equal units fill.
double wave_fill(double units, int sm_count) {
  const double waves = units / sm_count;
  return waves > 0 ? waves / std::ceil(waves) : 1.0;
}

// The part of a plan that the workspace depends on.
Plan plan_units(const moe_problem& p, int mode, int sm_count) {
  Plan pl{};
  const int K = (mode == MODE_SWIGLU) ? p.H : p.I;
  const int nslots = p.P + p.has_shared;
  const size_t out_cols = (mode == MODE_SWIGLU) ? p.I : p.H;
  pl.kb_total = (K + KB - 1) / KB;
  pl.pair = use_pairs(p, mode);
  const int ch = pl.pair ? 2 * BN : BN;  // token rows of one chunk at most
  const int workers = pl.pair ? sm_count / 2 : sm_count;
  // upper bound of the token chunks over all slots: a slot with rows has at least one of the
  // records, whose number bounds the chunks of a small batch
  const long records = (long)p.T * p.K + (long)p.has_shared * ((p.T + ch - 1) / ch);
  long chunks;
  if (p.layout == MOE_LAYOUT_MASKED) {
    chunks = (long)nslots * ((p.M_max + ch - 1) / ch);
  } else {
    const long rows = (long)p.T * p.K + (long)p.has_shared * p.T;
    chunks = std::min<long>((long)nslots * ((p.T + ch - 1) / ch), nslots + rows / ch);
  }
  chunks = std::min(chunks, records);
  // 128-row weight tiles; 64-row ones where they fill the SMs clearly better (one token of a
  // Mixtral-shaped layer: 224 pairs of 128-row gate/up tiles are 1.47 waves of 152 SMs)
  auto pairs_of = [&](int tw) { return (int)((mode == MODE_SWIGLU) ? p.I / tw : (p.H + 2 * tw - 1) / (2 * tw)); };
  pl.tw = 128;
  if (mode == MODE_SWIGLU && !pl.pair && chunks > 0 &&
      wave_fill((double)chunks * pairs_of(64), workers) > 1.1 * wave_fill((double)chunks * pairs_of(128), workers))
    pl.tw = 64;
  pl.pairs = pairs_of(pl.tw);
  const long tiles = chunks * pl.pairs;
  pl.ksplit = 1;
  if (mode == MODE_DOWN && !pl.pair && tiles > 0 && tiles < 3L * workers) {
    // split K so the unit count fills whole waves; at least four stages per split
    double best = 0.0;
    for (int ks = 1; ks <= 16 && pl.kb_total / ks >= 4; ++ks) {
      const double eff = wave_fill((double)tiles * ks, workers);
      if (eff > best + 0.02) {
        best = eff;
        pl.ksplit = ks;
      }
      if ((double)tiles * ks >= 2.0 * workers && eff >= 0.9) {
        pl.ksplit = ks;
        break;
      }
    }
  }
  auto split = [&](int ks) {
    pl.kb_per_split = (pl.kb_total + ks - 1) / ks;
    if (ks > 1) pl.kb_per_split = (pl.kb_per_split + GROUP - 1) / GROUP * GROUP;
    pl.ksplit = (pl.kb_total + pl.kb_per_split - 1) / pl.kb_per_split;
  };
  split(pl.ksplit);
  if (pl.ksplit > 1 && (size_t)pl.ksplit * grouped_rows(p) * out_cols * 4 > (size_t(1) << 30)) split(1);
  pl.part_bytes = pl.ksplit > 1 ? (size_t)pl.ksplit * grouped_rows(p) * out_cols * 4 : 0;
  return pl;
}

Plan make_plan(const moe_problem& p, int mode, int sm_count, int smem_cap) {
  Plan pl = plan_units(p, mode, sm_count);
  const int nslots = p.P + p.has_shared;
  const int stage = pl.pair ? Tile<128, true>::STAGE : pl.tw == 128 ? Tile<128, false>::STAGE : Tile<64, false>::STAGE;
  const int sf_buf = pl.tw == 128 ? Tile<128, false>::SF_BUF : Tile<64, false>::SF_BUF;
  for (int st = MAX_STAGES; st >= 2; --st) {
    size_t off = (size_t)st * stage;
    auto carve = [&](size_t bytes, size_t align) {
      off = align_up(off, align);
      const size_t at = off;
      off += bytes;
      return (uint32_t)at;
    };
    pl.sf_off = carve((size_t)SF_BUFS * sf_buf, 128);
    pl.pre_off = carve((3 * (size_t)nslots + 1) * 4, 16);
    pl.bar_off = carve((size_t)(2 * st + 4) * 8, 8);
    pl.misc_off = carve(16, 16);
    if ((int)(off + 1024) <= smem_cap) {
      pl.stages = st;
      pl.smem = off + 1024;
      break;
    }
  }
  return pl;
}

template <int MODE, int TW, bool PAIR, bool SPLIT>
int prepare_kernel() {
  auto kern = grouped_gemm_mx_kernel<MODE, TW, PAIR, SPLIT>;
  static bool attr_set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 64 && attr_set[dev]) return MOE_OK;
  // the register split must fit in what the launch provides, or setmaxnreg.inc would wait forever
  cudaFuncAttributes fa{};
  if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess) return MOE_ERR_CUDA;
  if (fa.numRegs * NUM_THREADS < SPLIT_REGS) return MOE_ERR_UNSUPPORTED;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, device_info().max_smem_optin) !=
      cudaSuccess)
    return MOE_ERR_CUDA;
  if (dev < 64) attr_set[dev] = true;
  return MOE_OK;
}

// Clusters of two that the device keeps resident at once (one CTA per SM), queried once per device and kernel.
template <int MODE>
int pair_clusters(size_t smem) {
  static int n[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 64 && n[dev] > 0) return n[dev];
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2 * (device_info().sm_count / 2));
  cfg.blockDim = dim3(NUM_THREADS);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int c = 0;
  if (cudaOccupancyMaxActiveClusters(&c, grouped_gemm_mx_kernel<MODE, 128, true, false>, &cfg) != cudaSuccess || c <= 0)
    return 0;
  c = std::min(c, device_info().sm_count / 2);
  if (dev < 64) n[dev] = c;
  return c;
}

template <int MODE, int TW, bool PAIR, bool SPLIT = false>
int launch_kernel(const Plan& pl, const CUtensorMap& tA, const TokenMaps& tB, const MxParams& prm, cudaStream_t st) {
  const int r = prepare_kernel<MODE, TW, PAIR, SPLIT>();
  if (r) return r;
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(NUM_THREADS);
  cfg.dynamicSmemBytes = pl.smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0] = overlap_attribute();
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (PAIR) {
    const int nc = pair_clusters<MODE>(pl.smem);
    if (nc <= 0) return MOE_ERR_CUDA;
    cfg.gridDim = dim3(2 * nc);
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  } else {
    cfg.gridDim = dim3(device_info().sm_count);
  }
  return cudaLaunchKernelEx(&cfg, grouped_gemm_mx_kernel<MODE, TW, PAIR, SPLIT>, tA, tB, prm) == cudaSuccess ? MOE_OK
                                                                                                    : MOE_ERR_CUDA;
}

}  // namespace

int gemm_mx_tile_rows(const moe_problem& p, int mode) { return use_pairs(p, mode) ? 2 * BN : BN; }

size_t gemm_mx_workspace_bytes(const moe_problem& p) {
  // the split (of the down product alone) depends on the SM count
  const size_t best = max_over_sm_counts([&](int sms) { return plan_units(p, MODE_DOWN, sms).part_bytes; });
  return STATS_BYTES + align_up(best, 256);
}

bool gemm_mx_splits(const moe_problem& p) { return plan_units(p, MODE_DOWN, device_info().sm_count).ksplit > 1; }

int launch_gemm_mx(const moe_problem& p, int mode, const void* act, const uint8_t* act_scales, const void* w,
                   const uint8_t* w_scales, const int32_t* masked_m, const int32_t* offsets, void* out,
                   uint8_t* out_scales, int32_t* err, void* ws, cudaStream_t st, const CombineArgs* comb,
                   bool after_gate_up) {
  const DeviceInfo& di = device_info();
  const Plan pl = make_plan(p, mode, di.sm_count, di.max_smem_optin);
  if (pl.stages == 0) return MOE_ERR_UNSUPPORTED;
  const int K = (mode == MODE_SWIGLU) ? p.H : p.I;
  const int NA = (mode == MODE_SWIGLU) ? 2 * p.I : p.H;
  const uint64_t rows = (uint64_t)grouped_rows(p);
  if (rows == 0) return MOE_OK;
  CUtensorMap tA;
  TokenMaps tB;
  if (encode_tensor_map(&tA, CU_TENSOR_MAP_DATA_TYPE_UINT8, K / 2, (uint64_t)(p.P + p.has_shared) * NA, K / 2,
                        ROW_BYTES, pl.tw, w) != CUDA_SUCCESS)
    return MOE_ERR_CUDA;
  // boxes for the rows that a chunk may have (the kernel takes no larger one, whatever the counts say)
  const int boxes = box_of((int)std::min<uint64_t>(p.layout == MOE_LAYOUT_MASKED ? p.M_max : rows, BN)) + 1;
  for (int i = 0; i < boxes; ++i)
    if (encode_tensor_map(&tB.box[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, K / 2, rows, K / 2, ROW_BYTES, box_rows(i), act) !=
        CUDA_SUCCESS)
      return MOE_ERR_CUDA;
  MxParams prm{};
  prm.mode = mode;
  prm.nslots = p.P + p.has_shared;
  prm.masked = p.layout == MOE_LAYOUT_MASKED;
  prm.M_max = p.M_max;
  prm.K = K;
  prm.kb_total = pl.kb_total;
  prm.kb_per_split = pl.kb_per_split;
  prm.ksplit = pl.ksplit;
  prm.NA = NA;
  prm.pairs = pl.pairs;
  prm.pair_stride = (mode == MODE_SWIGLU) ? pl.tw : 2 * pl.tw;
  prm.a1_off = (mode == MODE_SWIGLU) ? p.I : pl.tw;
  prm.out_cols = (mode == MODE_SWIGLU) ? p.I : p.H;
  prm.stages = pl.stages;
  prm.boxes = boxes;
  prm.early = after_gate_up;
  prm.vec_tok = K % 512 == 0 && (reinterpret_cast<uintptr_t>(act_scales) & 15u) == 0;
  prm.vec_w = K % 512 == 0 && (reinterpret_cast<uintptr_t>(w_scales) & 15u) == 0;
  prm.w_scales = w_scales;
  prm.act_scales = act_scales;
  prm.masked_m = masked_m;
  prm.offsets = offsets;
  prm.out = out;
  prm.out_scales = out_scales;
  prm.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + STATS_BYTES);
  prm.rows_total = (long)rows;
  prm.err = err;
  prm.stats = static_cast<int*>(ws);
  prm.sf_off = pl.sf_off;
  prm.pre_off = pl.pre_off;
  prm.bar_off = pl.bar_off;
  prm.misc_off = pl.misc_off;
  int r;
  if (mode == MODE_DOWN)
    r = pl.pair        ? launch_kernel<MODE_DOWN, 128, true>(pl, tA, tB, prm, st)
        : pl.ksplit > 1 ? launch_kernel<MODE_DOWN, 128, false, true>(pl, tA, tB, prm, st)
                        : launch_kernel<MODE_DOWN, 128, false>(pl, tA, tB, prm, st);
  else if (pl.pair)
    r = launch_kernel<MODE_SWIGLU, 128, true>(pl, tA, tB, prm, st);
  else
    r = pl.tw == 128 ? launch_kernel<MODE_SWIGLU, 128, false>(pl, tA, tB, prm, st)
                     : launch_kernel<MODE_SWIGLU, 64, false>(pl, tA, tB, prm, st);
  if (r) return r;
  return launch_splitk_reduce(p, prm.part, pl.ksplit, prm.out_cols, out, masked_m, offsets, st, comb, true);
}

}  // namespace moe
