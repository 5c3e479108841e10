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
// One CTA per SM, persistent.  A unit is (slot, chunk of at most 128 token rows, pair of 128-row
// weight tiles, K split); gate/up: the pair is the gate and the up tile of the same columns.
// Token rows are the MMA's M = 128 side and the pair its N = 256 side, so a token's row lies in
// one thread of the epilogue: SwiGLU, the MXFP4 form of h (a block is 32 columns of the row) and
// the stores are row-local.
//   * Warp 0: TMA producer.  A stage is 256 codes (128 bytes) of K: two weight tiles and the
//     token box (the smallest of 16 / 32 / 64 / 128 rows that covers the chunk).
//   * Warps 2-3: scale loaders.  Scales are row-major in global memory; the tensor core wants, for
//     128 rows and 128 codes, a 512-byte block with the four scale bytes of row r at
//     16 (r % 32) + 4 (r / 32).  A loader thread reads the 16 scale bytes of 512 codes of a row
//     and stores them as four words into the blocks of two stages (a group), one group ahead.
//   * Warp 1: one thread copies a stage's scale blocks from shared to tensor memory
//     (tcgen05.cp, which runs in order with the MMAs) and issues its four MMAs of K = 64.
//   * Warps 4-11: epilogue.  Columns 0-255 of tensor memory hold the unit's accumulators, the
//     columns above them the scales of the stages in flight.  The epilogue first moves the
//     accumulators to registers and hands them back, so only that move is not overlapped with
//     the next unit's MMAs; the copies run ahead through it.
//   * Every wait is bounded; on expiry the CTA drains its copies and MMAs, frees tensor memory,
//     reports MOE_FLAG_TIMEOUT and returns.
#include <algorithm>
#include <cmath>

#include "mx.cuh"

namespace moe {
namespace {

constexpr int STATS_CTAS = MOE_STATS_CTAS;
constexpr size_t STATS_BYTES = MOE_STATS_BYTES;
constexpr int BM = 128;                 // rows of one weight tile
constexpr int BN = 128;                 // token rows of one chunk at most
constexpr int ROW_BYTES = 128;          // bytes of a row in one stage (one 128-byte swizzle span)
constexpr int KB = 256;                 // codes of a row in one stage
constexpr int TILE_BYTES = 128 * ROW_BYTES;
constexpr int STAGE_BYTES = 3 * TILE_BYTES;  // weight tile 0 | weight tile 1 | tokens
constexpr int GROUP = 2;                // stages whose scales are loaded together (16 bytes of a row)
constexpr int SF_BLOCK = 512;           // scales of 128 rows and 128 codes
constexpr int SF_STAGE_TOK = 2 * SF_BLOCK;             // tokens: two blocks along K
constexpr int SF_STAGE_BYTES = SF_STAGE_TOK + 4 * SF_BLOCK;  // and the weights' two tiles of two blocks
constexpr int SF_RING = 3;              // groups of scales in flight
constexpr int SF_COLS = 24;             // tensor-memory columns of one stage's scales: 2 x 4 and 2 x 8
constexpr uint32_t SF_COL0 = 256;       // first of them
constexpr int NUM_THREADS = 384;
constexpr int EPI_THREADS = 256;
constexpr int EPI_WARP0 = 4;
constexpr int EPI_WARPS = EPI_THREADS / 32;
constexpr int LOAD_WARP0 = 2;
constexpr int LOAD_THREADS = 64;
// Register split (setmaxnreg): 4*32*ctrl + 8*32*epi <= 384 * (registers at launch), checked
// before the first launch.
constexpr int REGS_CTRL = 96, REGS_EPI = 200;
constexpr int REGS_NEEDED = 4 * 32 * REGS_CTRL + 8 * 32 * REGS_EPI;
constexpr uint32_t TMEM_COLS = 512;
constexpr long long TIMEOUT = 4000000000LL;  // SM cycles, about 2 s

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

struct Unit {
  int s, c, j, q;
  int nvalid;        // token rows of the chunk
  int rowB;          // first grouped-buffer row of the chunk
  int rowA0, rowA1;  // first weight row of each tile
  int kb0, kb1;      // stages
  bool a1;           // the second tile exists
};

__device__ __forceinline__ Unit decode_unit(const MxParams& p, const int* prefix, const int* srows, const int* sbase,
                                            int u) {
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
  const int nch = (m + BN - 1) / BN;
  U.q = r % p.ksplit;
  const int rest = r / p.ksplit;
  U.c = rest % nch;
  U.j = rest / nch;
  const int base = m / nch, extra = m - base * nch;  // near-equal chunks
  U.nvalid = base + (U.c < extra ? 1 : 0);
  U.rowB = sbase[lo] + U.c * base + min(U.c, extra);
  U.rowA0 = lo * p.NA + U.j * p.pair_stride;
  U.rowA1 = U.rowA0 + p.a1_off;
  U.a1 = p.mode == MODE_SWIGLU || U.j * p.pair_stride + p.a1_off < p.NA;
  U.kb0 = U.q * p.kb_per_split;
  U.kb1 = min(p.kb_total, U.kb0 + p.kb_per_split);
  return U;
}

// Shared-memory descriptor of a scale block: 32 rows of 16 bytes, no swizzle, 8-row groups 128
// bytes apart.
__device__ __forceinline__ uint64_t sf_desc(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(128 >> 4) << 32;  // stride byte offset
  d |= (uint64_t)1 << 46;           // descriptor version of the tcgen05 family
  return d;
}

// One scale block to four columns of tensor memory, repeated in its four lane quarters.
__device__ __forceinline__ void sf_copy(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// D[tmem] (+)= (A sfa) (B sfb)^T over K = 64 codes, issued by one thread.
__device__ __forceinline__ void mma_mxf4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                         uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n"
      "  .reg .pred p;\n"
      "  setp.ne.b32 p, %6, 0;\n"
      "  tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n"
      "}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

// Instruction descriptor of kind::mxf4: E2M1 x E2M1 with UE8M0 scales, K-major, M = 128; the
// scale factor id (0 or 2) picks the two bytes of a scale word that a K = 64 step uses.
__device__ __forceinline__ uint32_t mx_idesc(int N, uint32_t sf_id) {
  return (sf_id << 4)                   // B scale factor id
         | (1u << 7)                    // A: E2M1
         | (1u << 10)                   // B: E2M1
         | ((uint32_t)(N >> 3) << 17)   // N / 8
         | (1u << 23)                   // scales: UE8M0
         | ((uint32_t)(BM >> 4) << 24)  // M / 16
         | (sf_id << 29);               // A scale factor id
}

__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// n 32-byte vectors w(0..2n-1) (16 bytes each), as 32-byte stores when dst allows them.
template <int N, typename F>
__device__ __forceinline__ void store_row(uint8_t* dst, bool wide, F w) {
  if (wide) {
#pragma unroll
    for (int i = 0; i < N; ++i) st_global_v8(dst + 32 * i, w(2 * i), w(2 * i + 1));
  } else {
#pragma unroll
    for (int i = 0; i < 2 * N; ++i) reinterpret_cast<uint4*>(dst)[i] = w(i);
  }
}

template <int MODE>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    grouped_gemm_mx_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB16,
                           const __grid_constant__ CUtensorMap tmB32, const __grid_constant__ CUtensorMap tmB64,
                           const __grid_constant__ CUtensorMap tmB128, const MxParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* sf = smem + p.sf_off;                           // [SF_RING][GROUP][SF_STAGE_BYTES]
  int* prefix = reinterpret_cast<int*>(smem + p.pre_off);  // [nslots + 1] unit prefix
  int* srows = prefix + p.nslots + 1;                      // [nslots] valid rows per slot
  int* sbase = srows + p.nslots;                           // [nslots] first grouped-buffer row per slot
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + p.bar_off);
  uint64_t* empty = full + p.stages;
  uint64_t* sfull = empty + p.stages;    // [SF_RING] a group's scales stored
  uint64_t* sempty = sfull + SF_RING;    // [SF_RING] copied to tensor memory
  uint64_t* tfull = sempty + SF_RING;    // accumulators written
  uint64_t* tempty = tfull + 1;          // accumulators read
  uint64_t* drain = tempty + 1;
  uint32_t* tmem_base_smem = reinterpret_cast<uint32_t*>(smem + p.misc_off);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + p.misc_off + 4);

  const int tid = threadIdx.x;
  const int warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < SF_RING; ++i) {
      mbar_init(&sfull[i], LOAD_THREADS);
      mbar_init(&sempty[i], 1);
    }
    mbar_init(tfull, 1);
    mbar_init(tempty, EPI_WARPS);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_base_smem, TMEM_COLS);
    tmem_relinquish();
  }
  for (int s = tid; s < p.nslots; s += NUM_THREADS) {
    int m = __ldg(p.masked_m + s);
    if (p.masked) m = min(m, p.M_max);
    m = max(m, 0);
    srows[s] = m;
    sbase[s] = p.masked ? s * p.M_max : __ldg(p.offsets + s);
    prefix[s + 1] = (m + BN - 1) / BN * p.pairs * p.ksplit;
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
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_base_smem;
  const int total = prefix[p.nslots];

  if (warp < EPI_WARP0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_CTRL));
    if (warp == 0) {
      // ------------------------------------------------------------ producer
      if (lane == 0) {
        tma_prefetch_map(&tmA);
        tma_prefetch_map(&tmB16);
        tma_prefetch_map(&tmB32);
        tma_prefetch_map(&tmB64);
        tma_prefetch_map(&tmB128);
        const uint64_t pol = policy_evict_first();
        int stage = 0;
        uint32_t phase = 0;
        long issued = 0;
        bool ok = true;
        for (int u = blockIdx.x; ok && u < total; u += gridDim.x) {
          const Unit U = decode_unit(p, prefix, srows, sbase, u);
          const CUtensorMap* mb = &tmB128;
          int box = 128;
          if (U.nvalid <= 16) {
            mb = &tmB16;
            box = 16;
          } else if (U.nvalid <= 32) {
            mb = &tmB32;
            box = 32;
          } else if (U.nvalid <= 64) {
            mb = &tmB64;
            box = 64;
          }
          const uint32_t bytes = (U.a1 ? 2u : 1u) * TILE_BYTES + (uint32_t)box * ROW_BYTES;
          for (int kb = U.kb0; kb < U.kb1; ++kb) {
            if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, TIMEOUT)) {
              ok = false;
              break;
            }
            uint8_t* st = smem + (size_t)stage * STAGE_BYTES;
            const int x = kb * ROW_BYTES;
            mbar_arrive_expect_tx(&full[stage], bytes);
            tma_load_2d_hint(st, &tmA, &full[stage], x, U.rowA0, pol);
            if (U.a1) tma_load_2d_hint(st + TILE_BYTES, &tmA, &full[stage], x, U.rowA1, pol);
            tma_load_2d(st + 2 * TILE_BYTES, mb, &full[stage], x, U.rowB);
            ++issued;
            if (++stage == p.stages) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
        if (!ok) {
          // let the copies already in flight land before the CTA's shared memory is released
          const long first = issued > p.stages ? issued - p.stages : 0;
          for (long i = first; i < issued; ++i) {
            const int st = (int)(i % p.stages);
            const uint32_t ph = (uint32_t)((i / p.stages) & 1);
            const long long t0 = clock64();
            while (!mbar_try_wait(&full[st], ph) && clock64() - t0 < TIMEOUT) {
            }
          }
        }
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------ scale copies and MMAs
      if (lane == 0) {
        int stage = 0;
        uint32_t phase = 0, g_it = 0, u_it = 0;
        bool ok = true, any = false;
        int units = 0, tiles = 0;
        for (int u = blockIdx.x; ok && u < total; u += gridDim.x, ++u_it) {
          const Unit U = decode_unit(p, prefix, srows, sbase, u);
          ++units;
          tiles += (U.j == 0 && U.q == 0);  // one unit per (slot, token chunk)
          const int N = U.a1 ? 2 * BM : BM;
          const uint32_t id0 = mx_idesc(N, 0), id2 = mx_idesc(N, 2);
          if (!mbar_wait(tempty, (u_it & 1u) ^ 1u, abort_flag, TIMEOUT)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          uint32_t g = 0;
          for (int kb = U.kb0; kb < U.kb1; ++kb) {
            const int in_group = (kb - U.kb0) % GROUP;
            if (in_group == 0) {
              g = g_it % SF_RING;
              if (!mbar_wait(&sfull[g], (g_it / SF_RING) & 1u, abort_flag, TIMEOUT)) {
                ok = false;
                break;
              }
            }
            if (!mbar_wait(&full[stage], phase, abort_flag, TIMEOUT)) {
              ok = false;
              break;
            }
            tc_fence_after_sync();
            const int nk = min(4, (p.K - kb * KB) / 64);  // K = 64 steps of this stage: 4, or 2 at the end
            const uint32_t st = smem_u32(smem + (size_t)stage * STAGE_BYTES);
            const uint32_t ss = smem_u32(sf + (size_t)(g * GROUP + in_group) * SF_STAGE_BYTES);
            const uint32_t ta = tmem_base + SF_COL0 + (uint32_t)stage * SF_COLS, tb = ta + 8;
            const uint64_t dtok = smem_desc_sw128(st + 2 * TILE_BYTES), dw = smem_desc_sw128(st);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              if (2 * j < nk) {
                sf_copy(ta + 4 * j, sf_desc(ss + j * SF_BLOCK));
                sf_copy(tb + 8 * j, sf_desc(ss + SF_STAGE_TOK + (2 * j) * SF_BLOCK));
                if (U.a1) sf_copy(tb + 8 * j + 4, sf_desc(ss + SF_STAGE_TOK + (2 * j + 1) * SF_BLOCK));
                mma_mxf4(tmem_base, dtok + 4 * j, dw + 4 * j, id0, ta + 4 * j, tb + 8 * j, kb > U.kb0 || j > 0);
                mma_mxf4(tmem_base, dtok + 4 * j + 2, dw + 4 * j + 2, id2, ta + 4 * j, tb + 8 * j, 1u);
              }
            }
            any = true;
            tc_commit(&empty[stage]);
            if (in_group == GROUP - 1 || kb == U.kb1 - 1) {
              tc_commit(&sempty[g]);
              ++g_it;
            }
            if (++stage == p.stages) {
              stage = 0;
              phase ^= 1u;
            }
          }
          if (ok) tc_commit(tfull);
        }
        if (p.stats) {
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
        if (!ok && any) {
          // all MMAs issued by this thread must finish before tensor memory is freed
          tc_commit(drain);
          const long long t0 = clock64();
          while (!mbar_try_wait(drain, 0) && clock64() - t0 < TIMEOUT) {
          }
        }
      }
    } else {
      // ------------------------------------------------------------ scale loaders
      const int lt = tid - LOAD_WARP0 * 32;
      const int words = p.K / 128;             // words of a scale row
      const size_t row_bytes = (size_t)p.K / 32;
      // the 16 scale bytes of the codes from word w0 on (zeros past the row's end)
      auto fetch = [&](const uint8_t* row, int w0, bool vec) -> uint4 {
        if (vec) return __ldg(reinterpret_cast<const uint4*>(row) + (w0 >> 2));
        const uint32_t* w = reinterpret_cast<const uint32_t*>(row);
        return make_uint4(w0 < words ? __ldg(w + w0) : 0u, w0 + 1 < words ? __ldg(w + w0 + 1) : 0u,
                          w0 + 2 < words ? __ldg(w + w0 + 2) : 0u, w0 + 3 < words ? __ldg(w + w0 + 3) : 0u);
      };
      uint32_t g_it = 0;
      bool ok = true;
      for (int u = blockIdx.x; ok && u < total; u += gridDim.x) {
        const Unit U = decode_unit(p, prefix, srows, sbase, u);
        const uint8_t* rw0 = p.w_scales + (size_t)U.rowA0 * row_bytes;
        const uint8_t* rw1 = p.w_scales + (size_t)U.rowA1 * row_bytes;
        const uint8_t* rt = p.act_scales + (size_t)U.rowB * row_bytes;
        for (int kb = U.kb0; ok && kb < U.kb1; kb += GROUP, ++g_it) {
          const int w0 = kb * 2;
          uint4 vw[4], vt[2];
#pragma unroll
          for (int i = 0; i < 4; ++i) {  // rows lt, lt + 64 of tile 0, then of tile 1
            const int r = lt + 64 * (i & 1);
            vw[i] = make_uint4(0u, 0u, 0u, 0u);
            if (i < 2 || U.a1) vw[i] = fetch((i < 2 ? rw0 : rw1) + (size_t)r * row_bytes, w0, p.vec_w);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int r = lt + 64 * i;
            vt[i] = make_uint4(0u, 0u, 0u, 0u);
            if (r < U.nvalid) vt[i] = fetch(rt + (size_t)r * row_bytes, w0, p.vec_tok);
          }
          const uint32_t g = g_it % SF_RING;
          if (!mbar_wait(&sempty[g], ((g_it / SF_RING) & 1u) ^ 1u, abort_flag, TIMEOUT)) {
            ok = false;
            break;
          }
          uint8_t* dst = sf + (size_t)g * GROUP * SF_STAGE_BYTES;
          // word w of a row: stage w / 2 of the group, K block w % 2 of the stage
          auto put = [&](int block0, int block_step, int r, const uint4& v) {
            uint8_t* d = dst + block0 * SF_BLOCK + (r & 31) * 16 + (r >> 5) * 4;
            *reinterpret_cast<uint32_t*>(d) = v.x;
            *reinterpret_cast<uint32_t*>(d + block_step * SF_BLOCK) = v.y;
            *reinterpret_cast<uint32_t*>(d + SF_STAGE_BYTES) = v.z;
            *reinterpret_cast<uint32_t*>(d + SF_STAGE_BYTES + block_step * SF_BLOCK) = v.w;
          };
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            put(0, 1, lt + 64 * i, vt[i]);
            put(2, 2, lt + 64 * i, vw[i]);
            put(3, 2, lt + 64 * i, vw[2 + i]);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before tcgen05.cp reads them
          mbar_arrive(&sfull[g]);
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_EPI));
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3;              // tensor-memory lane quarter this warp may access
    const int half = (warp - EPI_WARP0) >> 2;  // column half of each tile
    const int lrow = quarter * 32 + lane;      // token row of this thread
    const uint32_t t_lane = tmem_base + ((uint32_t)(quarter * 32) << 16);
    const int c_lo = half * 64;
    const size_t oc = (size_t)p.out_cols;
    uint32_t u_it = 0;
    for (int u = blockIdx.x; u < total; u += gridDim.x, ++u_it) {
      const Unit U = decode_unit(p, prefix, srows, sbase, u);
      // the whole warp goes on together (its tensor-memory loads are warp-wide) or gives up together
      if (!__all_sync(0xffffffffu, mbar_wait(tfull, u_it & 1u, abort_flag, TIMEOUT))) break;
      tc_fence_after_sync();
      float acc0[64], acc1[64];
      const bool warp_live = quarter * 32 < U.nvalid;
      if (warp_live) {
#pragma unroll
        for (int pr = 0; pr < 2; ++pr) {
          float v0[32], v1[32];
          const uint32_t col = (uint32_t)(c_lo + pr * 32);
          tmem_ld32x2(t_lane + col, t_lane + col + 128u, v0, v1);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            acc0[pr * 32 + i] = v0[i];
            acc1[pr * 32 + i] = v1[i];
          }
        }
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(tempty);
      if (lrow >= U.nvalid) continue;  // rows past the chunk: nothing to store
      const size_t row = (size_t)(U.rowB + lrow);
      if constexpr (MODE == MODE_SWIGLU) {
#pragma unroll
        for (int i = 0; i < 64; ++i) acc0[i] = silu(acc0[i]) * acc1[i];
        uint32_t code[16], sb[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          float amax = 0.0f;
#pragma unroll
          for (int i = 0; i < 32; ++i) amax = mx_amax(amax, acc0[32 * b + i]);
          sb[b] = mx_scale_byte(amax);
          const float inv = mx_inv_scale(sb[b]);
#pragma unroll
          for (int i = 0; i < 4; ++i) code[4 * b + i] = mx_codes8(acc0 + 32 * b + 8 * i, inv);
        }
        const size_t col = (size_t)U.j * BM + c_lo;
        uint8_t* dst = static_cast<uint8_t*>(p.out) + row * (oc / 2) + col / 2;
        store_row<1>(dst, (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0, [&](int i) {
          return make_uint4(code[4 * i], code[4 * i + 1], code[4 * i + 2], code[4 * i + 3]);
        });
        *reinterpret_cast<uint16_t*>(p.out_scales + row * (oc / 32) + col / 32) = (uint16_t)(sb[0] | (sb[1] << 8));
      } else {
        const size_t col = (size_t)U.j * p.pair_stride + c_lo;
        if (p.ksplit > 1) {
          float* d = p.part + ((size_t)U.q * p.rows_total + row) * oc + col;
          const bool wide = (reinterpret_cast<uintptr_t>(p.part) & 31u) == 0;
          auto f4 = [](const float* a) {
            return [a](int i) {
              return make_uint4(__float_as_uint(a[4 * i]), __float_as_uint(a[4 * i + 1]), __float_as_uint(a[4 * i + 2]),
                                __float_as_uint(a[4 * i + 3]));
            };
          };
          store_row<8>(reinterpret_cast<uint8_t*>(d), wide, f4(acc0));
          if (U.a1) store_row<8>(reinterpret_cast<uint8_t*>(d + BM), wide, f4(acc1));
        } else {
          __nv_bfloat16* d = static_cast<__nv_bfloat16*>(p.out) + row * oc + col;
          const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0;
          auto h8 = [](const float* a) {
            return [a](int i) {
              return make_uint4(bf16x2(a[8 * i], a[8 * i + 1]), bf16x2(a[8 * i + 2], a[8 * i + 3]),
                                bf16x2(a[8 * i + 4], a[8 * i + 5]), bf16x2(a[8 * i + 6], a[8 * i + 7]));
            };
          };
          store_row<4>(reinterpret_cast<uint8_t*>(d), wide, h8(acc0));
          if (U.a1) store_row<4>(reinterpret_cast<uint8_t*>(d + BM), wide, h8(acc1));
        }
      }
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem_base, TMEM_COLS);
  }
  if (tid == 0 && *abort_flag) atomicOr(p.err, MOE_FLAG_TIMEOUT);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

struct Plan {
  int kb_total, kb_per_split, ksplit, pairs, stages;
  size_t smem, part_bytes;
  uint32_t sf_off, pre_off, bar_off, misc_off;
};

Plan make_plan(const moe_problem& p, int mode, int sm_count, int smem_cap) {
  Plan pl{};
  const int K = (mode == MODE_SWIGLU) ? p.H : p.I;
  const int nslots = p.P + p.has_shared;
  pl.kb_total = (K + KB - 1) / KB;
  pl.pairs = (mode == MODE_SWIGLU) ? p.I / BM : (p.H + 2 * BM - 1) / (2 * BM);
  // upper bound of the token chunks over all slots
  long chunks;
  if (p.layout == MOE_LAYOUT_MASKED) {
    chunks = (long)nslots * ((p.M_max + BN - 1) / BN);
  } else {
    const long rows = (long)p.T * p.K + (long)p.has_shared * p.T;
    chunks = std::min<long>((long)nslots * ((p.T + BN - 1) / BN), nslots + rows / BN);
  }
  const long tiles = chunks * pl.pairs;
  pl.ksplit = 1;
  if (mode == MODE_DOWN && tiles > 0 && tiles < 3L * sm_count) {
    // split K so the unit count fills whole waves; at least four stages per split
    double best = 0.0;
    for (int ks = 1; ks <= 16 && pl.kb_total / ks >= 4; ++ks) {
      const double waves = (double)(tiles * ks) / sm_count;
      const double eff = waves / std::ceil(waves);
      if (eff > best + 0.02) {
        best = eff;
        pl.ksplit = ks;
      }
      if (waves >= 2.0 && eff >= 0.9) {
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
  const size_t out_cols = (mode == MODE_SWIGLU) ? p.I : p.H;
  if (pl.ksplit > 1 && (size_t)pl.ksplit * grouped_rows(p) * out_cols * 4 > (size_t(1) << 30)) split(1);
  pl.part_bytes = pl.ksplit > 1 ? (size_t)pl.ksplit * grouped_rows(p) * out_cols * 4 : 0;
  for (int st = 6; st >= 2; --st) {
    size_t off = (size_t)st * STAGE_BYTES;
    auto carve = [&](size_t bytes, size_t align) {
      off = align_up(off, align);
      const size_t at = off;
      off += bytes;
      return (uint32_t)at;
    };
    pl.sf_off = carve((size_t)SF_RING * GROUP * SF_STAGE_BYTES, 128);
    pl.pre_off = carve((3 * (size_t)nslots + 1) * 4, 16);
    pl.bar_off = carve((size_t)(2 * st + 2 * SF_RING + 3) * 8, 8);
    pl.misc_off = carve(16, 16);
    if ((int)(off + 1024) <= smem_cap) {
      pl.stages = st;
      pl.smem = off + 1024;
      break;
    }
  }
  return pl;
}

template <int MODE>
int prepare_kernel() {
  auto kern = grouped_gemm_mx_kernel<MODE>;
  static bool attr_set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 64 && attr_set[dev]) return MOE_OK;
  // the register split must fit in what the launch provides, or setmaxnreg.inc would wait forever
  cudaFuncAttributes fa{};
  if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess) return MOE_ERR_CUDA;
  if (fa.numRegs * NUM_THREADS < REGS_NEEDED) return MOE_ERR_UNSUPPORTED;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, device_info().max_smem_optin) !=
      cudaSuccess)
    return MOE_ERR_CUDA;
  if (dev < 64) attr_set[dev] = true;
  return MOE_OK;
}

}  // namespace

int gemm_mx_tile_rows(const moe_problem&, int) { return BN; }

size_t gemm_mx_workspace_bytes(const moe_problem& p) {
  // the split depends on the SM count; sized for the largest plausible GPU (up to 256 SMs)
  size_t best = 0;
  for (int mode = 0; mode < 2; ++mode)
    for (int sms : {132, 148, 152, 160, 170, 188, 256}) best = std::max(best, make_plan(p, mode, sms, 232448).part_bytes);
  return STATS_BYTES + align_up(best, 256);
}

int launch_gemm_mx(const moe_problem& p, int mode, const void* act, const uint8_t* act_scales, const void* w,
                   const uint8_t* w_scales, const int32_t* masked_m, const int32_t* offsets, void* out,
                   uint8_t* out_scales, int32_t* err, void* ws, cudaStream_t st, const CombineArgs* comb) {
  const DeviceInfo& di = device_info();
  const Plan pl = make_plan(p, mode, di.sm_count, di.max_smem_optin);
  if (pl.stages == 0) return MOE_ERR_UNSUPPORTED;
  int r = mode == MODE_SWIGLU ? prepare_kernel<MODE_SWIGLU>() : prepare_kernel<MODE_DOWN>();
  if (r) return r;
  const int K = (mode == MODE_SWIGLU) ? p.H : p.I;
  const int NA = (mode == MODE_SWIGLU) ? 2 * p.I : p.H;
  const uint64_t rows = (uint64_t)grouped_rows(p);
  if (rows == 0) return MOE_OK;
  CUtensorMap tA, tB[4];
  if (encode_tensor_map(&tA, CU_TENSOR_MAP_DATA_TYPE_UINT8, K / 2, (uint64_t)(p.P + p.has_shared) * NA, K / 2,
                        ROW_BYTES, BM, w) != CUDA_SUCCESS)
    return MOE_ERR_CUDA;
  const int boxes[4] = {16, 32, 64, 128};
  for (int i = 0; i < 4; ++i)
    if (encode_tensor_map(&tB[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, K / 2, rows, K / 2, ROW_BYTES, boxes[i], act) !=
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
  prm.pair_stride = (mode == MODE_SWIGLU) ? BM : 2 * BM;
  prm.a1_off = (mode == MODE_SWIGLU) ? p.I : BM;
  prm.out_cols = (mode == MODE_SWIGLU) ? p.I : p.H;
  prm.stages = pl.stages;
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
  if (mode == MODE_SWIGLU)
    grouped_gemm_mx_kernel<MODE_SWIGLU><<<di.sm_count, NUM_THREADS, pl.smem, st>>>(tA, tB[0], tB[1], tB[2], tB[3], prm);
  else
    grouped_gemm_mx_kernel<MODE_DOWN><<<di.sm_count, NUM_THREADS, pl.smem, st>>>(tA, tB[0], tB[1], tB[2], tB[3], prm);
  if (cudaGetLastError() != cudaSuccess) return MOE_ERR_CUDA;
  return launch_splitk_reduce(p, prm.part, pl.ksplit, prm.out_cols, out, masked_m, offsets, st, comb);
}

}  // namespace moe
