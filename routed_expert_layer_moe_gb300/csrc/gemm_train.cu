// The products that train the experts (bf16), grouped by expert over ragged row counts.
//
//   UP   g, u = xg W13^T                 h = silu(g) u; g and u kept in 8 bits (e4m3, a scale per 128)
//   DH   dh = w dyg W2                   dg = dh u s (1 + g (1 - s)), du = dh g s, w h = w g s u, s = sigmoid(g),
//                                        with g and u as the checkpoint holds them, w the row's weight
//   DX   dxg = dgu W13                  in fp32: a token's rows of it are still added up
//   WG   dW[m][n] = sum over the rows of a slot of a[row][m] b[row][n]     (dW13 = dgu^T xg, dW2 = dyg^T (w h))
//
// Three launches: UP in the forward pass; DH and then DX with WG (GRAD), which need nothing of each other, in the backward
// pass.  One kernel form for all: clusters of two CTAs (SM pairs) whose tensor cores work on one tile of 256 x 256
// fp32 accumulators (cta_group::2, M = 256), each CTA staging 128 rows of either operand per 64 values of the reduced
// dimension: 32 KB a stage for 256 x 256 x 64 multiply-adds a pair.  Persistent; two accumulators in tensor
// memory, so a tile's epilogue runs beside the next tile's products.
//
// Every operand is read in the order it is stored, by TMA with the 128-byte swizzle:
//   * reduced dimension contiguous (xg, dyg, dgu, and W13 in UP): a stage is rows of 64 values, K-major.
//   * reduced dimension the outer one (W2 in DH, W13 in DX, both operands of WG): a stage is 64 rows of k with 64
//     columns in each of two boxes, MN-major; the tensor core transposes.
// So no weight is kept twice, and no operand is transposed in memory.
//
// Ragged rows.  Where the rows are the M side (UP, DH, DX), a chunk of up to 256 rows loads whole boxes: rows behind a
// slot's last one give accumulator rows that are not stored.  Where they are the reduced dimension (WG), the last 64 of
// a slot may hold rows of the next one, or padding, which may be NaN: MMAs of K = 16 stop behind the last row, and a
// warp writes zeros over the up to 15 rows between in shared memory, of both operands.  Such a last stage has a place of
// its own beside the ring of stages and is loaded early, so that the zeros are there when its turn comes; in the
// ring, the MMAs waited for them at the end of every tile (dW13 of 8 experts of 4096 x 14336, about 1024 rows each: 1330 us).
//
// Roles of a CTA: warp 0 TMA producer, warp 1 MMAs (leader CTA), warp 2 the zeros of WG, warps 4-11 epilogue.  Every
// wait is bounded; on expiry the CTA drains its copies and MMAs, frees tensor memory, reports MOE_FLAG_TIMEOUT and
// returns.
//
// What bounds it.  A stage moves 32 KB into each SM for 512 cycles of MMAs, 64 bytes a cycle: next to what the way from
// L2 gives, so operands are never staged twice and results leave without touching shared memory.  Long products run
// at 2.0 PFLOP/s for some milliseconds (dxg, 9728 rows of 4096 x 9728: 771 us) and at the power limit's clocks after
// that.  Experts' last chunks of less than 256 rows are whole tiles: 4.5 chunks for 1024 rows on average.  Measured (burst):
// 8 experts of 4096 x 14336, 4096 tokens of 2 records: UP 1090 to 1120 us (1.72 to 1.76 PFLOP/s), DH 610 to 650 (1.48 to
// 1.58), GRAD 2730 (1.76; DX alone, as a caller that wants no weights' gradients has it, 1140), with fp32 gradients 2970, added
// to what is there 4160; 64 experts of 2048 x 1024, 65536 rows: UP 360, DH 230 to 245, GRAD 845, fp32 920, added 1230; 512
// experts of 4096 x 1024, 160 rows each: UP 1400 to 1480 us, 6.5 to 6.7 TB/s.
#include <algorithm>
#include <type_traits>

#include "fp8.cuh"

namespace moe {
namespace {

enum { UP = 0, DH = 1, GRAD = 2 };     // launches; GRAD: DX and WG
enum { ROWS = 0, W13 = 1, W2 = 2 };    // what a unit is a tile of: rows' results (UP, DH, DX) or a gradient of weights

constexpr int KB = 64;                    // reduced values of a stage: 128 bytes of a K-major row
constexpr int HALF = 128;                 // rows of an operand that one CTA stages
constexpr int OP_BYTES = HALF * KB * 2;   // one operand of a stage
constexpr int BOX_BYTES = OP_BYTES / 2;   // MN-major: 64 k rows of 64 columns
constexpr int STAGE = 2 * OP_BYTES;
constexpr int MAX_STAGES = 6;
constexpr int THREADS = 384;
constexpr int EPI_WARP0 = 4, EPI_WARPS = 8;
constexpr uint32_t TMEM_COLS = 512, ACC_COLS = 256;
constexpr int GROUP_M = 8;                // M tiles that neighbouring units share an N tile with
constexpr long long TIMEOUT = 4000000000LL;  // SM cycles, about 2 s
// GRAD: stages from which on lanes store their own rows.  Short tiles are bound by their stores, which want whole lines
// (dW13 + dW2 of 64 rows, 4864 x 4096: 22.9 + 15.7 us own, 19.5 + 12.2 exchanged; 512 rows 35 + 21, 33.5 + 20); beside long
// ones the exchange's shuffles take shared memory's cycles from the MMAs (1024 rows: 51.6 + 29.0 own, 54 + 30 exchanged).
constexpr int OWN_ROWS_KB = 12;
constexpr int NUM_BOXES = 3;              // row boxes of 32, 64 and 128
__host__ __device__ constexpr int box_rows(int i) { return 32 << i; }
__host__ __device__ constexpr int box_of(int rows) { return rows <= 32 ? 0 : rows <= 64 ? 1 : 2; }

struct Maps {
  CUtensorMap a[NUM_BOXES];  // rows, by box
  CUtensorMap b;             // weights
  CUtensorMap wa[2], wb[2];  // GRAD: operands of dW13 and dW2
};

struct WeightGrad {    // dW [slots][rows][cols]
  int rows, cols;
  int mt, nt, units;   // tiles; units of a slot: mt * nt, or 0 where the gradient is not wanted
  uint64_t group_inv;  // ceil(2^64 / (GROUP_M nt))
  void* out;
};

struct Params {
  int nslots, masked, M_max;
  long long rows_total;
  int kb;              // UP, DH, DX: stages of the reduced dimension
  int nt;              // N tiles; GRAD: 0 where dxg is not wanted
  uint64_t group_inv;  // ceil(2^64 / (GROUP_M nt))
  int b_rows;          // rows of one slot in the weights
  int ncols;           // columns of the output: UP, DH: I; DX: H
  WeightGrad w[2];     // GRAD
  int stages;
  int accumulate;      // dW, fp32: add to what is there
  int wide;            // the outputs are 32-byte aligned
  const int32_t* masked_m;
  const int32_t* offsets;
  void* out;           // UP, DH: h (DH: times w) bf16 [rows][I]; DX: dxg fp32 [rows][H]
  void* out2;          // UP: codes [rows][2 I]; DH: dgu bf16 [rows][2 I]
  float* out2_s;       // UP: scales [rows][2 I / 128]
  const uint8_t* gu;   // DH: codes and scales of the checkpoint
  const float* gu_s;
  const float* wg;     // DH: weights of the rows, or null
  int32_t* err;
  uint32_t ex_off, pre_off, bar_off, misc_off;
};

struct Unit {
  int kind, slot, mi, j;  // slot, chunk of rows (weights: M tile), N tile
  int row;                // first row of this CTA's part of the chunk; weights: first row of the slot
  int nvalid, nall;       // rows of this CTA's part, of both parts; weights: rows of the slot
  int kb;                 // stages
};

// ceil(2^32 / n) for n = 2 .. GROUP_M: r / n = umulhi(r, it) for r < 2^29.
__constant__ uint32_t kInverse[9] = {0,          0,          0x80000000u, 0x55555556u, 0x40000000u,
                                               0x33333334u, 0x2AAAAAABu, 0x24924925u, 0x20000000u};

// The slots of a launch in shared memory, by place (GRAD: by descending row count, else their own order).
struct Slots {
  int *prefix, *wprefix;  // units before a place: of rows, of weights (GRAD)
  int *rows, *base;       // rows, first row
  int* order;             // GRAD: the slot at a place
};

// A role's walk over its units.  The place is carried along and nothing is divided on the way: a look-up stands between
// the last copies or products of one unit and the first of the next.
//
// Units of rows, all of one cost, are dealt in rounds over the pairs of CTAs.  GRAD goes on with those of weights, the
// most rows first: to the pairs that the last, partial round of rows left out as many as one unit of rows is worth,
// then to all, every other round backwards, so that the sums of what each is dealt differ by little (64 experts with 200
// to 4000 rows: the longest 1.01 to 1.05 of the mean; 1.07 to 1.3 in the slots' own order, always forwards).
template <int MODE>
struct Walk {
  const Params& p;
  const Slots& s;
  uint32_t rank;
  int i, pairs;           // this pair of CTAs among all
  int wtotal, mine;       // units of weights; units of rows that are this pair's
  int first, nlag, ahead, extra;  // pairs from `first` on, nlag of them, get `ahead` units of weights; this one gets `extra`
  int place, round, u;
  bool weights;

  __device__ __forceinline__ Walk(const Params& p_, const Slots& s_, uint32_t rank_)
      : p(p_), s(s_), rank(rank_), i((int)cluster_id_x()), pairs((int)nclusters_x()), place(0), round(0), weights(false) {
    const int total = s.prefix[p.nslots], whole = total / pairs;
    first = total - whole * pairs;
    mine = whole + (i < first);
    wtotal = nlag = ahead = extra = 0;
    if constexpr (MODE == GRAD) {
      wtotal = s.wprefix[p.nslots];
      if (first > 0) {
        nlag = pairs - first;
        ahead = (p.kb + 3) / ((s.rows[0] + KB - 1) / KB + 3);  // a tile costs about three stages beside its own
        if (i >= first) extra = ahead;
      }
    }
  }

  // Goes on to the next unit, number u of its kind; false behind the last.
  __device__ __forceinline__ bool next() {
    int k = round++;
    if (k < mine) {
      u = k * pairs + i;
      return true;
    }
    if constexpr (MODE != GRAD) return false;
    if (!weights) {
      weights = true;
      place = 0;
    }
    k -= mine;
    if (k < extra) {
      u = k * nlag + i - first;
    } else {
      k -= extra;
      u = ahead * nlag + k * pairs + (k & 1 ? pairs - 1 - i : i);
    }
    return u < wtotal;
  }

  __device__ __forceinline__ void seek() {
    const int* prefix = MODE == GRAD && weights ? s.wprefix : s.prefix;
    while (prefix[place + 1] <= u) ++place;
  }

  __device__ __forceinline__ Unit unit() {
    seek();
    Unit U;
    U.slot = MODE == GRAD ? s.order[place] : place;
    const int m = s.rows[place];
    int r = u, nm, nt;
    uint64_t inv;
    if (MODE == GRAD && weights) {
      r -= s.wprefix[place];
      U.kind = r < p.w[0].units ? W13 : W2;
      if (U.kind == W2) r -= p.w[0].units;
      const WeightGrad& w = p.w[U.kind - W13];
      nm = w.mt, nt = w.nt, inv = w.group_inv;
    } else {
      r -= s.prefix[place];
      U.kind = ROWS;
      nm = (m + 2 * HALF - 1) / (2 * HALF), nt = p.nt, inv = p.group_inv;
    }
    // groups of GROUP_M tiles of M, the M tile the fastest within one: a wave of pairs shares operands through L2
    const int group = (int)__umul64hi((uint64_t)r, inv) * GROUP_M;
    const int size = min(GROUP_M, nm - group), rr = r - group * nt;
    U.j = size == 1 ? rr : (int)__umulhi((uint32_t)rr, kInverse[size]);
    U.mi = group + rr - U.j * size;
    if (U.kind != ROWS) {
      U.row = s.base[place];
      U.nvalid = U.nall = m;
      U.kb = (m + KB - 1) / KB;
    } else {
      // whole parts of 128 rows as far as they go
      U.nall = min(2 * HALF, m - U.mi * 2 * HALF);
      U.nvalid = rank ? max(U.nall - HALF, 0) : min(U.nall, HALF);
      U.row = s.base[place] + U.mi * 2 * HALF + (int)rank * HALF;
      U.kb = p.kb;
    }
    return U;
  }
};

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

__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n"
      "  .reg .pred p;\n"
      "  setp.ne.b32 p, %4, 0;\n"
      "  tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n"
      "}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Arrival on an mbarrier of the cluster that other CTAs' reads of this CTA's shared memory are ordered by.
__device__ __forceinline__ void arrive_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// Shared-memory matrix descriptor of an MN-major tile: boxes of 64 k rows x 128 bytes (64 columns) written with the
// 128-byte swizzle.  Eight k rows are 1024 bytes (stride byte offset), the next 64 columns a box further (leading one).
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)(BOX_BYTES >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// a_mn, b_mn: the operand is MN-major.
__host__ __device__ constexpr uint32_t instruction_desc(bool a_mn, bool b_mn) {
  return mma_idesc<false>(2 * HALF, 2 * HALF) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u);
}

__device__ __forceinline__ void tmem_load32(uint32_t taddr, float (&v)[32]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
                 "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
               : "r"(taddr)
               : "memory");
}

// Wait for this thread's loads from tensor memory; v is what one of them wrote.
__device__ __forceinline__ void tmem_loaded32(float (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]),
                 "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31])
               :
               : "memory");
}

// N (32 or 64) columns of this thread's lane of tensor memory.
template <int N>
__device__ __forceinline__ void tmem_load(uint32_t taddr, float (&v)[N]) {
  float a[32];
  tmem_load32(taddr, a);
  if constexpr (N == 64) {
    float b[32];
    tmem_load32(taddr + 32, b);
    tmem_loaded32(b);
#pragma unroll
    for (int i = 0; i < 32; ++i) v[32 + i] = b[i];
  }
  tmem_loaded32(a);
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = a[i];
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Transposes pieces of eight words among L = N / 8 neighbouring lanes: piece j of lane i of them becomes piece i of lane j.
template <int N>
__device__ __forceinline__ void exchange_pieces(uint32_t (&v)[N], int lane) {
  constexpr int L = N / 8;
#pragma unroll
  for (int d = 1; d < L; d *= 2) {
    const bool up = lane & d;
#pragma unroll
    for (int j = 0; j < L; ++j)
      if (!(j & d)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          uint32_t &lo = v[8 * j + i], &hi = v[8 * (j + d) + i];
          const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? lo : hi, d);
          if (up)
            lo = got;
          else
            hi = got;
        }
      }
  }
}

// N words of each lane's row to memory, without shared memory: through it, coalesced or by TMA, the stores take cycles
// of it from the MMAs, whose operands come from there at half its rate.  A lane storing its own row would touch 32 lines
// an instruction (4.3 TB/s for whole tiles, 5.4 with whole lines); so L = N / 8 lanes first exchange their pieces of 32
// bytes, after which each holds one piece of L rows, and L lanes store 32 L bytes of a row together.
// first: the warp's first row; rows: how many of the 32 are written; add: to the fp32 values there; wide: 32-byte aligned.
// own: without the exchange.
template <int N>
__device__ __forceinline__ void store_rows(void* first, size_t stride, int lane, uint32_t (&v)[N], int rows, bool wide,
                                           bool add = false, bool own = false) {
  constexpr int L = N / 8;
  if (!own) exchange_pieces(v, lane);
  // piece j of the lane: of row r0 + j, or of the lane's own row
  const int r0 = own ? lane : lane / L * L;
  const size_t step = own ? 32 : stride;
  uint8_t* at = static_cast<uint8_t*>(first) + (size_t)r0 * stride + (own ? 0 : 32 * (lane % L));
#pragma unroll
  for (int j = 0; j < L; ++j) {
    if (r0 + (own ? 0 : j) < rows) {
      uint4* q = reinterpret_cast<uint4*>(at + j * step);
      uint32_t* x = &v[8 * j];
      if (add) {
        const float4 f = reinterpret_cast<const float4*>(q)[0], g = reinterpret_cast<const float4*>(q)[1];
        const float old[8] = {f.x, f.y, f.z, f.w, g.x, g.y, g.z, g.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) + old[i]);
      }
      const uint4 a = make_uint4(x[0], x[1], x[2], x[3]), b = make_uint4(x[4], x[5], x[6], x[7]);
      if (wide) {
        st_global_v8(q, a, b);
      } else {
        q[0] = a;
        q[1] = b;
      }
    }
  }
}

// 128 columns of a warp's 32 accumulator rows to memory; zero: zeros in their place.
template <typename OUT>
__device__ __forceinline__ void store_tile(OUT* first, int cols, int lane, uint32_t acc, int rows, bool zero, bool add,
                                           bool wide, bool own) {
  constexpr int COLS = 128 / sizeof(OUT);  // 128 bytes of a row at a time
#pragma unroll 1
  for (int c = 0; c < HALF; c += COLS) {
    uint32_t v[32];
    if (zero) {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = 0u;
    } else {
      float d[COLS];
      tmem_load<COLS>(acc + (uint32_t)c, d);
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = sizeof(OUT) == 2 ? pack2(d[(2 * i) % COLS], d[(2 * i + 1) % COLS]) : __float_as_uint(d[i]);
    }
    store_rows(first + c, (size_t)cols * sizeof(OUT), lane, v, rows, wide, sizeof(OUT) == 4 && add, own);
  }
}

// DH: what a lane's row needs beside the accumulator: weight, scales, and the codes of 32 columns of g and u.  Requested
// before the tile's products are waited for, and 32 columns ahead (dh of 64 experts of 2048 x 1024: 231 -> 227 us).
struct Kept {
  float w, sg, su;
  uint4 g[2], u[2];
};

__device__ __forceinline__ void fetch_codes(Kept& k, const uint8_t* code, int I) {
  k.g[0] = __ldg(reinterpret_cast<const uint4*>(code));
  k.g[1] = __ldg(reinterpret_cast<const uint4*>(code) + 1);
  k.u[0] = __ldg(reinterpret_cast<const uint4*>(code + I));
  k.u[1] = __ldg(reinterpret_cast<const uint4*>(code + I) + 1);
}

// The lane's row and first column in a tile of DH; false: the warp has nothing to do.
__device__ __forceinline__ bool dh_place(const Params& p, const Unit& U, int ew, int lane, size_t& row, int& c0) {
  c0 = U.j * 2 * HALF + HALF * (ew >> 2);
  const int rows = U.nvalid - 32 * (ew & 3);
  row = (size_t)U.row + 32 * (ew & 3) + (lane < rows ? lane : 0);  // a lane without a row reads the warp's first
  return c0 < p.ncols && rows > 0;
}

__device__ __forceinline__ void dh_begin(const Params& p, const Unit& U, int ew, int lane, Kept& k) {
  size_t row;
  int c0;
  if (!dh_place(p, U, ew, lane, row, c0)) return;
  const int I = p.ncols, n = 2 * I / FP8_GROUP;
  k.w = p.wg ? p.wg[row] : 1.0f;
  k.sg = p.gu_s[row * n + c0 / FP8_GROUP];
  k.su = p.gu_s[row * n + (I + c0) / FP8_GROUP];
  fetch_codes(k, p.gu + row * 2 * I + c0, I);
}

// The epilogue of one tile, warp `ew` of the eight: lanes 32 (ew & 3) .. of the CTA's 128 accumulator rows, columns
// 128 (ew >> 2) .. of its 256 (UP: 64 of the gate's and the same 64 of the up's).  acc: the warp's lanes and the
// tile's first column; `zero`: there is no accumulator, the tile is zeros (dW of a slot without rows).
template <int MODE, typename OUT>
__device__ __forceinline__ void epilogue(const Params& p, const Unit& U, uint32_t rank, int ew, int lane, uint32_t acc,
                                         float* ex, bool zero, Kept& kept) {
  const int quad = ew & 3, half = ew >> 2;
  const int r = 32 * quad + lane;  // the lane's row in the CTA's 128
  if constexpr (MODE == UP) {
    const int I = p.ncols, c0 = U.j * HALF + 64 * half;
    float g[32], u[32];
    float ag = 0.0f, au = 0.0f;
#pragma unroll
    for (int c = 0; c < 64; c += 32) {
      tmem_load32(acc + 64 * half + c, g);
      tmem_load32(acc + HALF + 64 * half + c, u);
      tmem_loaded32(g);
      tmem_loaded32(u);
#pragma unroll
      for (int i = 0; i < 32; ++i) ag = fp8_amax(ag, g[i]), au = fp8_amax(au, u[i]);
    }
    // a group's other 64 columns are with the warp of the same rows in the other half
    reinterpret_cast<float2*>(ex)[half * HALF + r] = make_float2(ag, au);
    asm volatile("bar.sync %0, 64;" ::"r"(1 + quad) : "memory");
    if (U.nvalid <= 32 * quad) return;
    const float2 other = reinterpret_cast<float2*>(ex)[(half ^ 1) * HALF + r];
    const float sg = fp8_scale(fp8_amax(ag, other.x)), su = fp8_scale(fp8_amax(au, other.y));
    // one division a group; the codes' inputs are fp32 sums, so a reciprocal's last bit is within their own error
    // (scales whose reciprocal would overflow: both sides times 2^100)
    const bool tiny_g = sg < 0x1p-100f, tiny_u = su < 0x1p-100f;
    const float ig = 1.0f / (tiny_g ? sg * 0x1p100f : sg), iu = 1.0f / (tiny_u ? su * 0x1p100f : su);
    const size_t row = (size_t)U.row + r;
    if (half == 0 && r < U.nvalid) {
      p.out2_s[row * (2 * I / FP8_GROUP) + U.j] = sg;
      p.out2_s[row * (2 * I / FP8_GROUP) + I / FP8_GROUP + U.j] = su;
    }
    const int rows = U.nvalid - 32 * quad;
    const size_t row0 = (size_t)U.row + 32 * quad;
    uint32_t qg[16], qu[16];
#pragma unroll
    for (int c = 0; c < 64; c += 32) {
      tmem_load32(acc + 64 * half + c, g);
      tmem_load32(acc + HALF + 64 * half + c, u);
      tmem_loaded32(g);
      tmem_loaded32(u);
      uint32_t h[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) h[i] = pack2(silu(g[2 * i]) * u[2 * i], silu(g[2 * i + 1]) * u[2 * i + 1]);
      if (tiny_g) {
#pragma unroll
        for (int i = 0; i < 32; ++i) g[i] *= 0x1p100f;
      }
      if (tiny_u) {
#pragma unroll
        for (int i = 0; i < 32; ++i) u[i] *= 0x1p100f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {  // a group without a scale has codes 0
        qg[c / 4 + i] = sg != sg ? 0u : fp8_pair(g[4 * i] * ig, g[4 * i + 1] * ig) | fp8_pair(g[4 * i + 2] * ig, g[4 * i + 3] * ig) << 16;
        qu[c / 4 + i] = su != su ? 0u : fp8_pair(u[4 * i] * iu, u[4 * i + 1] * iu) | fp8_pair(u[4 * i + 2] * iu, u[4 * i + 3] * iu) << 16;
      }
      store_rows(static_cast<__nv_bfloat16*>(p.out) + row0 * I + c0 + c, (size_t)I * 2, lane, h, rows, p.wide);
    }
    uint8_t* code = static_cast<uint8_t*>(p.out2) + row0 * 2 * I + c0;
    store_rows(code, (size_t)I * 2, lane, qg, rows, p.wide);
    store_rows(code + I, (size_t)I * 2, lane, qu, rows, p.wide);
  } else if constexpr (MODE == DH) {
    const int I = p.ncols, rows = U.nvalid - 32 * quad;
    size_t row;
    int c0;
    if (!dh_place(p, U, ew, lane, row, c0)) return;
    const size_t row0 = (size_t)U.row + 32 * quad;
    const float w = kept.w, sg = kept.sg, su = kept.su;
    const uint8_t* code = p.gu + row * 2 * I + c0;
    __nv_bfloat16* dgu = static_cast<__nv_bfloat16*>(p.out2) + row0 * 2 * I + c0;
    __nv_bfloat16* hg = static_cast<__nv_bfloat16*>(p.out) + row0 * I + c0;
#pragma unroll 1
    for (int c = 0; c < HALF; c += 32) {
      const uint32_t qg[8] = {kept.g[0].x, kept.g[0].y, kept.g[0].z, kept.g[0].w,
                              kept.g[1].x, kept.g[1].y, kept.g[1].z, kept.g[1].w};
      const uint32_t qu[8] = {kept.u[0].x, kept.u[0].y, kept.u[0].z, kept.u[0].w,
                              kept.u[1].x, kept.u[1].y, kept.u[1].z, kept.u[1].w};
      if (c + 32 < HALF) fetch_codes(kept, code + c + 32, I);
      float d[32];
      tmem_load32(acc + HALF * half + (uint32_t)c, d);
      tmem_loaded32(d);
      uint32_t vg[16], vu[16], vh[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float2 cg = fp8_unpair(qg[i >> 1] >> (16 * (i & 1))), cu = fp8_unpair(qu[i >> 1] >> (16 * (i & 1)));
        float dg[2], du[2], h[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float g = (e ? cg.y : cg.x) * sg, u = (e ? cu.y : cu.x) * su, x = w * d[2 * i + e];
          const float s = __fdividef(1.0f, 1.0f + __expf(-g));
          const float gs = g * s;
          h[e] = w * (gs * u);
          du[e] = x * gs;
          dg[e] = x * u * fmaf(gs, 1.0f - s, s);
        }
        vg[i] = pack2(dg[0], dg[1]);
        vu[i] = pack2(du[0], du[1]);
        vh[i] = pack2(h[0], h[1]);
      }
      store_rows(dgu + c, (size_t)I * 4, lane, vg, rows, p.wide);
      store_rows(dgu + I + c, (size_t)I * 4, lane, vu, rows, p.wide);
      store_rows(hg + c, (size_t)I * 2, lane, vh, rows, p.wide);
    }
  } else {
    const int c0 = U.j * 2 * HALF + HALF * half;
    acc += HALF * half;
    const bool own = U.kb >= OWN_ROWS_KB;
    if (U.kind == ROWS) {
      const int rows = U.nvalid - 32 * quad;
      if (c0 < p.ncols && rows > 0)
        store_tile(static_cast<float*>(p.out) + ((size_t)U.row + 32 * quad) * p.ncols + c0, p.ncols, lane, acc, rows,
                   false, false, p.wide, own);
    } else {
      const WeightGrad& w = p.w[U.kind - W13];
      const int m = U.mi * 2 * HALF + (int)rank * HALF;  // whole tiles of 128 rows and columns
      if (c0 < w.cols && m < w.rows)
        store_tile(static_cast<OUT*>(w.out) + ((size_t)U.slot * w.rows + m + 32 * quad) * w.cols + c0, w.cols, lane, acc,
                   32, zero, p.accumulate, p.wide, own);
    }
  }
}

// Whether both warps that meet at hardware barrier `id` (64 threads) are ok.
__device__ __forceinline__ bool both_ok(int id, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n"
      "  .reg .pred p, q;\n"
      "  setp.ne.b32 q, %1, 0;\n"
      "  bar.red.and.pred p, %2, 64, q;\n"
      "  selp.u32 %0, 1, 0, p;\n"
      "}\n"
      : "=r"(r)
      : "r"((uint32_t)ok), "r"(id)
      : "memory");
  return r;
}

template <int MODE, typename OUT>
__global__ void __launch_bounds__(THREADS, 1)
    train_gemm_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
  float* ex = reinterpret_cast<float*>(smem + p.ex_off);   // UP: [2 tiles][2 halves][128 rows] (gate, up) magnitudes
  Slots S;
  S.prefix = reinterpret_cast<int*>(smem + p.pre_off);
  S.rows = S.prefix + p.nslots + 1;
  S.base = S.rows + p.nslots;
  S.order = S.base + p.nslots;
  S.wprefix = S.order + p.nslots;  // GRAD: [nslots + 1]
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + p.bar_off);
  uint64_t* empty = full + MAX_STAGES;
  uint64_t* landed = empty + MAX_STAGES;  // weights, the last stage that needs zeros: this CTA's copies are there
  uint64_t* fixed = landed + 1;           // both CTAs have written the zeros
  uint64_t* last_empty = fixed + 1;       // the MMAs have read it
  uint64_t* tfull = last_empty + 1;       // [2] accumulators written
  uint64_t* tempty = tfull + 2;           // [2] read
  uint64_t* drain = tempty + 2;
  uint64_t* fin = drain + 1;              // the peer CTA is done with this CTA's memory
  uint32_t* tmem_base_smem = reinterpret_cast<uint32_t*>(smem + p.misc_off);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + p.misc_off + 4);

  const int tid = threadIdx.x;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int stages = p.stages;

  if (tid == 0) {
    for (int i = 0; i < MAX_STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(landed, 1);
    mbar_init(fixed, 2);
    mbar_init(last_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], 2 * EPI_WARPS);
    }
    mbar_init(drain, 1);
    mbar_init(fin, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc<true>(tmem_base_smem, TMEM_COLS);
    tmem_relinquish<true>();
  }
  // launched while the kernel before it in the stream may still run: nothing global is read or written before this
  grid_dependency_wait();
  grid_dependents_launch();
  for (int s = tid; s < p.nslots; s += THREADS) {
    long long base = p.masked ? (long long)s * p.M_max : (long long)__ldcg(p.offsets + s);
    int m = __ldcg(p.masked_m + s);
    if (p.masked) m = min(m, p.M_max);
    if (base < 0 || base > p.rows_total) base = p.rows_total;  // no counts may lead outside the buffers
    m = (int)max(0LL, min((long long)m, p.rows_total - base));
    if constexpr (MODE == GRAD) {
      S.order[s] = m;  // the row counts, until they are in order
    } else {
      S.rows[s] = m;
      S.base[s] = (int)base;
      S.prefix[s + 1] = (m + 2 * HALF - 1) / (2 * HALF) * p.nt;
    }
  }
  if constexpr (MODE == GRAD) {
    __syncthreads();
    int place[3];  // of this thread's slots: there are at most 1024
    int i = 0;
    for (int s = tid; s < p.nslots; s += THREADS, ++i) {
      const int m = S.order[s];
      int n = 0;
      for (int t = 0; t < p.nslots; ++t) n += S.order[t] > m || (S.order[t] == m && t < s);
      place[i] = n;
      S.rows[n] = m;
      S.prefix[n + 1] = (m + 2 * HALF - 1) / (2 * HALF) * p.nt;
      S.wprefix[n + 1] = m == 0 && p.accumulate ? 0 : p.w[0].units + p.w[1].units;
    }
    __syncthreads();
    i = 0;
    for (int s = tid; s < p.nslots; s += THREADS, ++i) {
      S.order[place[i]] = s;
      const long long base = p.masked ? (long long)s * p.M_max : (long long)__ldcg(p.offsets + s);
      S.base[place[i]] = (int)(base < 0 || base > p.rows_total ? p.rows_total : base);
    }
  }
  if (tid == 0) S.prefix[0] = 0;
  if (MODE == GRAD && tid == 0) S.wprefix[0] = 0;
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 0 || (MODE == GRAD && warp == 1)) {
    int* prefix = warp == 0 ? S.prefix : S.wprefix;
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
  cluster_sync_all();  // both CTAs' barriers are initialised before either CTA touches the other's
  tc_fence_after_sync();
  const uint32_t tmem_base = __shfl_sync(0xffffffffu, *tmem_base_smem, 0);
  Walk<MODE> walk(p, S, rank);
  // rows of a slot's last stage that are in its last MMA's 16 but behind the last row
  auto ragged = [](const Unit& U) { return MODE == GRAD && U.kind != ROWS && (U.nvalid & 15) != 0; };

  if (warp == 0) {
    // -------------------------------------------------------------- producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, lphase = 0;
      bool ok = true;
      while (ok && walk.next()) {
        const Unit U = walk.unit();
        const bool weights = MODE == GRAD && U.kind != ROWS;
        const CUtensorMap* ma = weights ? &maps.wa[U.kind - W13] : &maps.a[box_of(U.nvalid)];
        const CUtensorMap* mb = weights ? &maps.wb[U.kind - W13] : &maps.b;
        auto row_bytes = [](int rows) { return rows > 0 ? (uint32_t)box_rows(box_of(rows)) * KB * 2 : 0u; };
        // of both CTAs; a part without rows copies none, but zeros in UP
        const uint32_t bytes = weights || MODE == UP
                                   ? 2 * STAGE
                                   : row_bytes(min(U.nall, HALF)) + row_bytes(U.nall - HALF) + 2 * OP_BYTES;
        const int am = U.mi * 2 * HALF + (int)rank * HALF;
        const int bn = U.j * (MODE == UP ? HALF : 2 * HALF) + (MODE == UP ? 0 : (int)rank * HALF);
        const int brow = weights ? U.row : U.slot * p.b_rows + (MODE == UP ? (int)rank * p.ncols + bn : 0);
        const int whole = ragged(U) ? U.kb - 1 : U.kb;  // stages that go through the ring
        for (int kb = 0; ok && kb <= whole; ++kb) {
          // the last stage's place is free at the latest when the ring has gone round once in this tile
          if (whole < U.kb && kb == min(whole, stages)) {
            if (!mbar_wait(last_empty, lphase ^ 1u, abort_flag, TIMEOUT)) {
              ok = false;
              break;
            }
            lphase ^= 1u;
            mbar_arrive_expect_tx(landed, STAGE);  // counted here: warp 2 has to see this CTA's copies land
            uint8_t* sa = smem + (size_t)stages * STAGE;
            const int y = U.row + whole * KB;
            for (int h = 0; h < 2; ++h) {
              tma_load_2d(sa + h * BOX_BYTES, ma, landed, am + 64 * h, y);
              tma_load_2d(sa + OP_BYTES + h * BOX_BYTES, mb, landed, bn + 64 * h, y);
            }
          }
          if (kb == whole) break;
          if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, TIMEOUT)) {
            ok = false;
            break;
          }
          uint8_t* sa = smem + (size_t)stage * STAGE;
          uint8_t* sb = sa + OP_BYTES;
          const int k = kb * KB;
          // the leader's barrier counts both CTAs' copies
          if (leader) mbar_arrive_expect_tx(&full[stage], bytes);
          const uint32_t bar = mapa_shared(&full[stage], 0);
          if (weights) {
            for (int h = 0; h < 2; ++h) tma_load_2d_pair(sa + h * BOX_BYTES, ma, bar, am + 64 * h, U.row + k);
          } else {
            // The box that holds the part's rows.  UP: and zeros behind it (boxes behind the buffer's end, which read
            // nothing): MMAs of zeros draw less power than those of what a stage held before, which long runs are bound
            // by (8 experts of 4096 x 14336: 1368 -> 1354 us; the gradient's products, whose stages turn over faster,
            // lost 2% by it).
            const int have = U.nvalid > 0 ? box_rows(box_of(U.nvalid)) : 0;
            const int end = (int)p.rows_total;
            if (have > 0) tma_load_2d_pair(sa, ma, bar, k, U.row);
            if constexpr (MODE == UP) {
              if (have == 0) tma_load_2d_pair(sa, &maps.a[2], bar, k, end);
              if (have == 32) tma_load_2d_pair(sa + 32 * KB * 2, &maps.a[0], bar, k, end);
              if (have == 32 || have == 64) tma_load_2d_pair(sa + 64 * KB * 2, &maps.a[1], bar, k, end);
            }
          }
          if constexpr (MODE == UP) {
            tma_load_2d_pair(sb, mb, bar, k, brow);
          } else {
            for (int h = 0; h < 2; ++h) tma_load_2d_pair(sb + h * BOX_BYTES, mb, bar, bn + 64 * h, brow + k);
          }
          if (++stage == stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    }
  } else if (warp == 1) {
    // -------------------------------------------------------------- MMAs: a converged warp, one elected lane
    const uint32_t s0 = smem_u32(smem);
    int stage = 0;
    uint32_t phase = 0, fphase = 0, it = 0;
    bool ok = true, any = false;
    // The MMAs of a unit of nkb stages.  WEIGHTS: of a slot's `rows`, the reduced dimension.  The two kinds are code of
    // their own, so that all that an MMA takes but the stage is a constant.
    auto products = [&](auto weights_, int nkb, int rows) {
      constexpr bool WEIGHTS = decltype(weights_)::value;
      const uint64_t da0 = WEIGHTS ? desc_mn(s0) : smem_desc_sw128(s0);
      const uint64_t db0 = MODE == UP ? smem_desc_sw128(s0 + OP_BYTES) : desc_mn(s0 + OP_BYTES);
      // 16 values of k: 32 bytes of a K-major row, 16 rows of an MN-major box
      constexpr uint32_t STEP_K = 2, STEP_MN = 16 * 128 / 16;
      constexpr uint32_t STEP_A = WEIGHTS ? STEP_MN : STEP_K, STEP_B = MODE == UP ? STEP_K : STEP_MN;
      constexpr uint32_t idesc = instruction_desc(WEIGHTS, MODE != UP);
      const uint32_t d = tmem_base + (it & 1u) * ACC_COLS;
      ok = __all_sync(0xffffffffu, mbar_wait<true>(&tempty[it & 1u], ((it >> 1) & 1u) ^ 1u, abort_flag, TIMEOUT));
      if (!ok) return;
      tc_fence_after_sync();
      // one stage's MMAs, of `steps` times 16 values of k
      auto multiply = [&](int at, int steps, bool first, uint64_t* done) {
        tc_fence_after_sync();
        const uint64_t da = da0 + (uint32_t)at * (STAGE >> 4), db = db0 + (uint32_t)at * (STAGE >> 4);
        if (elect_one()) {
#pragma unroll
          for (int ks = 0; ks < KB / 16; ++ks)
            if (!WEIGHTS || ks < steps) mma_pair(d, da + ks * STEP_A, db + ks * STEP_B, idesc, !first || ks > 0);
          tc_commit_pair(done, 3);
        }
        __syncwarp();
        any = true;
      };
      const int whole = WEIGHTS && (rows & 15) ? nkb - 1 : nkb;
      for (int kb = 0; kb < whole; ++kb) {
        ok = __all_sync(0xffffffffu, mbar_wait<true>(&full[stage], phase, abort_flag, TIMEOUT));
        if (!ok) return;
        multiply(stage, WEIGHTS && kb == nkb - 1 ? (rows - kb * KB) / 16 : KB / 16, kb == 0, &empty[stage]);
        if (++stage == stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (WEIGHTS && whole < nkb) {
        ok = __all_sync(0xffffffffu, mbar_wait<true>(fixed, fphase, abort_flag, TIMEOUT));
        if (!ok) return;
        fphase ^= 1u;
        multiply(stages, (rows - whole * KB + 15) / 16, whole == 0, last_empty);
      }
      if (elect_one()) tc_commit_pair(&tfull[it & 1u], 3);
      __syncwarp();
      ++it;
    };
    while (ok && leader && walk.next()) {
      if (MODE != GRAD || !walk.weights) {
        products(std::false_type{}, p.kb, 0);
      } else {
        walk.seek();
        const int rows = __shfl_sync(0xffffffffu, S.rows[walk.place], 0);
        if (rows > 0) products(std::true_type{}, (rows + KB - 1) / KB, rows);
      }
    }
    if (!ok && any && elect_one()) {
      // all MMAs issued by this thread must finish before tensor memory is freed
      tc_commit_pair(drain, 1);
      const long long t0 = clock64();
      while (!mbar_try_wait(drain, 0) && clock64() - t0 < TIMEOUT) {
      }
    }
    __syncwarp();
  } else if (warp == 2) {
    // -------------------------------------------------------------- weights: zeros behind a slot's last row
    if constexpr (MODE == GRAD) {
      uint32_t lphase = 0;
      while (walk.next()) {
        if (!walk.weights) continue;
        walk.seek();
        const int m = S.rows[walk.place];
        if ((m & 15) == 0) continue;
        // the first of these waits lasts through all units of rows: 16 limits, about half a minute
        if (!__all_sync(0xffffffffu, mbar_wait(landed, lphase, abort_flag, 16 * TIMEOUT))) break;
        lphase ^= 1u;
        const int v = m % KB, n = 16 - (v & 15);  // rows v .. v + n - 1 of the stage
        uint8_t* at = smem + (size_t)stages * STAGE + v * 128;
        for (int i = lane; i < n * 8 * 4; i += 32)  // eight 16-byte pieces a row, four boxes
          *reinterpret_cast<uint4*>(at + (i & 3) * BOX_BYTES + (i >> 2) * 16) = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_shared();  // the tensor cores read them
        __syncwarp();
        if (lane == 0) arrive_cluster(mapa_shared(fixed, 0));
      }
    }
  } else if (warp >= EPI_WARP0) {
    // -------------------------------------------------------------- epilogue
    const int ew = warp - EPI_WARP0;
    uint32_t it = 0;
    while (walk.next()) {
      const Unit U = walk.unit();
      if (MODE == GRAD && U.kb == 0) {
        Kept none;
        epilogue<MODE, OUT>(p, U, rank, ew, lane, 0u, ex, true, none);
        continue;
      }
      Kept kept;
      if constexpr (MODE == DH) dh_begin(p, U, ew, lane, kept);
      const uint32_t b = it & 1u;
      bool ok = __all_sync(0xffffffffu, mbar_wait<true>(&tfull[b], (it >> 1) & 1u, abort_flag, TIMEOUT));
      if constexpr (MODE == UP) ok = both_ok(1 + (ew & 3), ok);  // the two warps of a row go on or give up together
      if (!ok) break;
      tc_fence_after_sync();
      const uint32_t acc = tmem_base + b * ACC_COLS + ((uint32_t)(32 * (ew & 3)) << 16);
      epilogue<MODE, OUT>(p, U, rank, ew, lane, acc, ex + b * 4 * HALF, false, kept);
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(mapa_shared(&tempty[b], 0));
      ++it;
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  // Neither CTA frees its tensor memory or leaves while the other may still use it: the leader's MMAs read the peer's
  // shared memory and write its tensor memory, the peer's copies and arrivals land on the leader's barriers.
  if (tid == 0) {
    if (*abort_flag) {  // let copies in flight land before shared memory is released
      const uint64_t t0 = global_timer_ns();
      while (global_timer_ns() - t0 < 200000u) {
      }
    }
    mbar_arrive_remote(mapa_shared(fin, rank ^ 1u));
    const long long t0 = clock64();
    while (!mbar_try_wait<true>(fin, 0)) {
      if (clock64() - t0 > TIMEOUT) {
        *abort_flag = 1;
        break;
      }
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc<true>(tmem_base, TMEM_COLS);
  }
  if (tid == 0 && *abort_flag) atomicOr(p.err, MOE_FLAG_TIMEOUT);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

// Shared memory of a launch: as many stages as fit, but one less in GRAD, whose last stages have a place of their own:
// what a launch leaves of the SM's memory is the L1 that stores go through (dW13 + dW2 of 64 experts of 2048 x 1024:
// 380 + 209 us with six and that place, 370 + 196 with five).
int lay_out(Params& prm, int mode, size_t* smem) {
  for (int st = mode == GRAD ? MAX_STAGES - 1 : MAX_STAGES; st >= 2; --st) {
    size_t off = (size_t)(mode == GRAD ? st + 1 : st) * STAGE;  // GRAD: and the place of a slot's last stage
    auto carve = [&](size_t bytes, size_t align) {
      off = align_up(off, align);
      const size_t at = off;
      off += bytes;
      return (uint32_t)at;
    };
    prm.ex_off = carve(mode == UP ? 2 * 2 * HALF * 2 * sizeof(float) : 0, 16);
    prm.pre_off = carve((5 * (size_t)prm.nslots + 2) * 4, 16);
    prm.bar_off = carve((2 * MAX_STAGES + 9) * 8, 8);
    prm.misc_off = carve(16, 16);
    if ((int)(off + 1024) <= device_info().max_smem_optin) {
      prm.stages = st;
      *smem = off + 1024;
      return MOE_OK;
    }
  }
  return MOE_ERR_UNSUPPORTED;
}

void cluster_attribute(cudaLaunchAttribute* a) {
  a->id = cudaLaunchAttributeClusterDimension;
  a->val.clusterDim.x = 2;
  a->val.clusterDim.y = 1;
  a->val.clusterDim.z = 1;
}

template <int MODE, typename OUT>
int launch(Params prm, const Maps& maps, cudaStream_t st) {
  prm.wide = 1;
  for (const void* q : {(const void*)prm.out, (const void*)prm.out2, (const void*)prm.w[0].out, (const void*)prm.w[1].out})
    if (reinterpret_cast<uintptr_t>(q) & 31u) prm.wide = 0;
  auto kern = train_gemm_kernel<MODE, OUT>;
  static bool attr_set[64] = {};
  static int clusters[64] = {};  // clusters of two that the device keeps resident at once
  size_t smem = 0;
  const int r = lay_out(prm, MODE, &smem);
  if (r) return r;
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) return MOE_ERR_UNSUPPORTED;
  if (!attr_set[dev]) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, device_info().max_smem_optin) !=
        cudaSuccess)
      return MOE_ERR_CUDA;
    attr_set[dev] = true;
  }
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  cluster_attribute(&attr[0]);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (clusters[dev] == 0) {
    cfg.gridDim = dim3(2 * (device_info().sm_count / 2));
    int c = 0;
    if (cudaOccupancyMaxActiveClusters(&c, kern, &cfg) != cudaSuccess || c <= 0) return MOE_ERR_CUDA;
    clusters[dev] = std::min(c, device_info().sm_count / 2);
  }
  cfg.gridDim = dim3(2 * clusters[dev]);
  attr[1] = overlap_attribute();
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, maps, prm) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

bool map_of(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, uint32_t box) {
  return encode_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, cols, rows, cols * 2, KB, box, base) == CUDA_SUCCESS;
}

Params common_params(const moe_problem& p, const int32_t* masked_m, const int32_t* offsets, int32_t* err) {
  Params prm{};
  prm.nslots = p.P + p.has_shared;
  prm.masked = p.layout == MOE_LAYOUT_MASKED;
  prm.M_max = p.M_max;
  prm.rows_total = grouped_rows(p);
  prm.masked_m = masked_m;
  prm.offsets = offsets;
  prm.err = err;
  return prm;
}

// ceil(2^64 / (GROUP_M nt)): the divisor is at least 8, so it does not overflow.
uint64_t group_inverse(int nt) { return nt ? ~0ull / ((uint64_t)GROUP_M * nt) + 1 : 0; }

// Rows of the M side [rows][K] times the weights [slots][b_rows][b_cols].
int plan_rows(int mode, Params& prm, Maps& maps, const void* a, int K, const void* w, int b_rows, int b_cols, int ncols) {
  for (int i = 0; i < NUM_BOXES; ++i)
    if (!map_of(&maps.a[i], a, K, (uint64_t)prm.rows_total, box_rows(i))) return MOE_ERR_CUDA;
  if (!map_of(&maps.b, w, b_cols, (uint64_t)prm.nslots * b_rows, mode == UP ? HALF : KB)) return MOE_ERR_CUDA;
  prm.kb = K / KB;
  prm.b_rows = b_rows;
  prm.ncols = ncols;
  prm.nt = mode == UP ? ncols / HALF : (ncols + 2 * HALF - 1) / (2 * HALF);
  prm.group_inv = group_inverse(prm.nt);
  return MOE_OK;
}

// a [rows][M], b [rows][N] -> dw [slots][M][N].
int plan_weights(Params& prm, Maps& maps, int i, const void* a, int M, const void* b, int N, void* dw) {
  if (!map_of(&maps.wa[i], a, M, (uint64_t)prm.rows_total, KB) || !map_of(&maps.wb[i], b, N, (uint64_t)prm.rows_total, KB))
    return MOE_ERR_CUDA;
  WeightGrad& w = prm.w[i];
  w.rows = M;
  w.cols = N;
  w.mt = (M + 2 * HALF - 1) / (2 * HALF);
  w.nt = (N + 2 * HALF - 1) / (2 * HALF);
  w.units = w.mt * w.nt;
  w.group_inv = group_inverse(w.nt);
  w.out = dw;
  return MOE_OK;
}

}  // namespace

int launch_swiglu_save(const moe_problem& p, const void* xg, const void* w13, const int32_t* masked_m,
                       const int32_t* offsets, void* hg, uint8_t* gu, float* gu_scales, int32_t* err,
                       cudaStream_t st) {
  if (grouped_rows(p) == 0) return MOE_OK;
  Params prm = common_params(p, masked_m, offsets, err);
  prm.out = hg;
  prm.out2 = gu;
  prm.out2_s = gu_scales;
  Maps maps{};
  const int r = plan_rows(UP, prm, maps, xg, p.H, w13, 2 * p.I, p.H, p.I);
  return r ? r : launch<UP, __nv_bfloat16>(prm, maps, st);
}

int launch_ffn_backward(const moe_problem& p, const FfnBackwardArgs& a, cudaStream_t st) {
  const Params prm = common_params(p, a.masked_m, a.offsets, a.err);
  const size_t nslots = prm.nslots, es = a.dw_dtype == MOE_F32 ? 4 : 2;
  if (prm.rows_total == 0) {  // no rows: the weights' gradients are zeros
    for (void* dw : {a.dw13, a.dw2}) {
      const size_t n = nslots * p.H * p.I * (dw == a.dw13 ? 2 : 1) * es;
      if (dw && !a.accumulate && cudaMemsetAsync(dw, 0, n, st) != cudaSuccess) return MOE_ERR_CUDA;
    }
    return MOE_OK;
  }
  Params dh = prm;
  dh.out = a.hg;
  dh.out2 = a.dgu;
  dh.gu = a.gu;
  dh.gu_s = a.gu_scales;
  dh.wg = a.wg;
  Maps maps{};
  int r = plan_rows(DH, dh, maps, a.dyg, p.H, a.w2, p.H, p.I, p.I);
  if (!r) r = launch<DH, __nv_bfloat16>(dh, maps, st);
  if (r || !(a.dxg || a.dw13 || a.dw2)) return r;
  Params g = prm;
  g.out = a.dxg;
  g.accumulate = a.accumulate;
  if (a.dxg) r = plan_rows(GRAD, g, maps, a.dgu, 2 * p.I, a.w13, 2 * p.I, p.H, p.H);
  if (!r && a.dw13) r = plan_weights(g, maps, 0, a.dgu, 2 * p.I, a.xg, p.H, a.dw13);
  if (!r && a.dw2) r = plan_weights(g, maps, 1, a.dyg, p.H, a.hg, p.I, a.dw2);
  if (r) return r;
  return a.dw_dtype == MOE_F32 ? launch<GRAD, float>(g, maps, st) : launch<GRAD, __nv_bfloat16>(g, maps, st);
}

}  // namespace moe
