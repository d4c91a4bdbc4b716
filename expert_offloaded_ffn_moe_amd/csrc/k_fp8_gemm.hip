// Product of e4m3 codes with a scale for each block of 128, for many tokens: tiles of tokens x
// channels through a ring of LDS buffers, a block of 128 of K a step.
//
//   out[t][n] = sum_b (sx[t][b] sw[n / 128][b]) sum_{k in b} x[t][k] w[n][k] + ...
//
// Tokens are the row operand and channels the column operand of a 16 x 16 MFMA, so a lane
// receives the sums of column l % 16 and rows 4 (l / 16) .. + 3. A block's sum starts from zero and
// is added to the tile's with its scales, 4 multiply-adds for each 16 x 16 x 128 product, beside
// which the matrix pipe goes on.
//
// bf16 outputs take v_mfma_f32_16x16x128_f8f6f4 on the codes themselves, 32 of a row a lane. It
// adds eight neighbouring products at a time, each cut to 2^-13 of the binade of the largest
// (measured with one large product beside small ones), and those sums in fp32: of normal codes the
// outputs are off by 1.5e-5, of codes of every size alike by 2^-13 of the sum of the products' sizes,
// and never by more than 7 x 2^-13 of it. That is under the outputs' own rounding of 2^-8 unless
// they nearly cancel. It is taken for its rate: the bf16 MFMA, on which the products are exact, has
// half of it and its operands have to be converted first (2048 x 7168 x 7168 250 us in fp32, 121 so; 256 x
// 7168 43 and 31; 64 x 7168 20.1 and 19.5). fp32 outputs take that one, four steps of 32 a block.
//
// LDS holds rows of 128 bytes, whose 16-byte pieces stand at places piece ^ (row / 2 % 8), so that
// the lanes that a read serves at once use every bank once; loads go from memory to LDS
// directly, in lane order, so that each lane fetches the piece that belongs at its place. Lane
// quarter q reads pieces q and 4 + q of both operands. Pieces past K come from a line of
// zeros. Scales follow the same way, a wave's part of the rows' and its channels' one, those of
// four steps at once: a row's scales are neighbours, and their line comes from L2 once for them.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "f8_dev.h"
#include "fp8.h"
#include "int8_out.h"
#include "tiles.h"

namespace moe {
namespace {

typedef int32_t i32x8 __attribute__((ext_vector_type(8)));

constexpr int kBK = kF8Block;  // bytes of a row in a step

__device__ __forceinline__ int swizzle(int r) { return (r >> 1) & 7; }

__device__ const f8i4 zero_codes = {0, 0, 0, 0};

// A row's (column's) 32 codes of a lane, and as four operands of the bf16 MFMA.
struct Codes {
  i32x8 v;
};
struct Converted {
  bf16x8v v[4];
};
template <bool EXACT>
struct Operand {
  typedef Codes T;
  static __device__ __forceinline__ T of(const Codes& c) { return c; }
};
template <>
struct Operand<true> {
  typedef Converted T;
  static __device__ __forceinline__ T of(const Codes& c) {
    T t;
#pragma unroll
    for (int i = 0; i < 4; ++i) t.v[i] = f8_to_bf16(c.v[2 * i], c.v[2 * i + 1]);
    return t;
  }
};
__device__ __forceinline__ f32x4 block_product(const Codes& x, const Codes& w) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x.v, w.v, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ f32x4 block_product(const Converted& x, const Converted& w) {
  f32x4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) p = mfma_bf16(x.v[i], w.v[i], p);
  return p;
}

// Four neighbouring channels of PASSES rows, ROWS apart, from their sums in LDS (of PARTS parts,
// PART floats apart). WHOLE: every row and channel is one of the matrix's, and what the rows
// need is loaded for all of them before it is used.
template <bool BF16, int PASSES, int ROWS, int LDROW, int PARTS, int PART, bool WHOLE>
__device__ __forceinline__ void store_rows(const Fp8Args& a, int64_t t0, int n, const float* from, const float* bias) {
  typedef typename OutElem<BF16>::T E;
  constexpr int kAt = PASSES < 4 ? PASSES : 4;  // rows at once
  const int left = WHOLE ? 4 : a.N - n;
  if (!WHOLE && left <= 0) return;
#pragma unroll
  for (int p0 = 0; p0 < PASSES; p0 += kAt) {
    float v[kAt][4], more[kAt][4];
#pragma unroll
    for (int p = 0; p < kAt; ++p) {
      const int r = (p0 + p) * ROWS;
      f32x4 s = *reinterpret_cast<const f32x4*>(from + r * LDROW);
#pragma unroll
      for (int k = 1; k < PARTS; ++k) s += *reinterpret_cast<const f32x4*>(from + k * PART + r * LDROW);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[p][e] = s[e] + bias[e];
    }
    if (a.o.y) {
#pragma unroll
      for (int p = 0; p < kAt; ++p)
        if (WHOLE || t0 + (p0 + p) * ROWS < a.T) load4(a.o.y + (t0 + (p0 + p) * ROWS) * a.o.ld_y + n, left, more[p]);
#pragma unroll
      for (int p = 0; p < kAt; ++p)
#pragma unroll
        for (int e = 0; e < 4; ++e) v[p][e] += more[p][e];
    }
    if (a.o.res) {
#pragma unroll
      for (int p = 0; p < kAt; ++p)
        if (WHOLE || t0 + (p0 + p) * ROWS < a.T)
          load4(static_cast<const E*>(a.o.res) + (t0 + (p0 + p) * ROWS) * a.o.ld_res + n, left, more[p]);
#pragma unroll
      for (int p = 0; p < kAt; ++p)
#pragma unroll
        for (int e = 0; e < 4; ++e) v[p][e] += more[p][e];
    }
#pragma unroll
    for (int p = 0; p < kAt; ++p)
      if (WHOLE || t0 + (p0 + p) * ROWS < a.T)
        store4(static_cast<E*>(a.o.out) + (t0 + (p0 + p) * ROWS) * a.o.ld_out + n, left, v[p]);
  }
}

// WM x WN waves, each 32 TM x 32 TN; RING buffers. KG such groups of waves take the blocks of K in
// turn, each with buffers of its own, and add their sums at the end.
//
// A step's rows and columns are in registers when it starts. Early in it (when its last reads are
// sure to be in) the waves meet: the buffer that they were read from is filled anew, and the next
// one, which is full, is read, into the registers of each block of rows after its products and a
// second set of columns. Both are spread over the rest of the step, since all waves' reads
// together take LDS as long as the products take.
template <int WM, int WN, int TM, int TN, int RING, int KG, bool BF16>
__global__ __launch_bounds__(64 * WM* WN* KG) void k_fp8_gemm(Fp8Args a, int mtiles) {
  typedef Operand<!BF16> Make;
  typedef typename Make::T Op;
  constexpr int kWaves = WM * WN, BM = 32 * TM * WM, BN = 32 * TN * WN;
  constexpr int kLoadsA = BM / 8 / kWaves, kLoadsB = BN / 8 / kWaves, kLoads = kLoadsA + kLoadsB;  // of a wave per step, of 8 rows
  static_assert(kLoadsA * 8 * kWaves == BM && kLoadsB * 8 * kWaves == BN, "rows divide among the waves");
  constexpr int kOwnRows = BM / kWaves, kOwn = kOwnRows + 4;  // rows whose scales a wave loads; its floats in LDS
  static_assert(kOwnRows % 4 == 0 && kOwnRows < 64, "a lane for each row and one for the channels");
  constexpr int kSteps = 4;  // whose scales are loaded together
  __shared__ __attribute__((aligned(1024))) uint8_t all[KG][RING][(BM + BN) * kBK];
  __shared__ __attribute__((aligned(16))) float all_scales[KG][2][kSteps][kWaves * kOwn];
  const int lane = threadIdx.x & 63, wave_id = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = KG == 1 ? 0 : wave_id / kWaves, wave = KG == 1 ? wave_id : wave_id % kWaves;
  auto& sh = all[group];
  const int tile = xcd_order(blockIdx.x, gridDim.x);
  const int m0 = tile % mtiles * BM, n0 = tile / mtiles * BN;
  const int wm = wave / WN, wn = wave % WN, l16 = lane & 15, quarter = lane >> 4;
  const int blocks = f8_blocks(a.K);

  // this lane's piece of each row that it fetches; rows past the last are read as the last,
  // and not stored
  const uint8_t* p[kLoads];
  int at[kLoads];  // its offset in K
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const bool in_a = i < kLoadsA;
    const int r = (in_a ? wave * kLoadsA + i : wave * kLoadsB + i - kLoadsA) * 8 + lane / 8;
    const int64_t row = in_a ? min(m0 + r, a.T - 1) : min(n0 + r, a.N - 1);
    at[i] = ((lane % 8) ^ swizzle(r)) * 16;
    p[i] = (in_a ? a.x + row * a.ld_x : a.w + row * a.ld_w) + group * kBK + at[i];
  }
  const float* scales = lane < kOwnRows ? a.sx + (int64_t)min(m0 + wave * kOwnRows + lane, a.T - 1) * a.ld_sx
                                        : a.sw + (int64_t)(min(n0 + wn * 32 * TN, a.N - 1) / kF8Block) * a.ld_sw;
  const uint8_t* zeros = reinterpret_cast<const uint8_t*>(&zero_codes);
  const uint32_t ring = (uint32_t)(uintptr_t)(lvoid*)&sh[0][0], scale_sets = (uint32_t)(uintptr_t)(lvoid*)&all_scales[group][0][0][0];
  int kat = group;  // the next block to load
  // the scales of the next kSteps steps into set `set`, past the last block 0
  auto stage_scales = [&](int set) {
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      const void* scale = kat + k * KG < blocks ? (const void*)(scales + kat + k * KG) : zeros;
      if (lane <= kOwnRows) load_one_to_lds(scale, scale_sets + ((set * kSteps + k) * kWaves + wave) * kOwn * 4);
    }
  };
  // the part'th of `parts` parts of the next step's loads, into buffer `buf` (past the last block: zeros)
  auto stage = [&](int buf, int part, int parts) {
    const uint32_t to = ring + buf * (uint32_t)sizeof(sh[0]);
    if (part == 0) {
      if ((kat + 1) * kBK > a.K) {  // the last of K is in it, or nothing
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
          if (kat * kBK + at[i] >= a.K) p[i] = zeros;
      }
      kat += KG;
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      if (i < kLoads * part / parts || i >= kLoads * (part + 1) / parts) continue;
      load_to_lds(p[i], to + (i < kLoadsA ? (wave * kLoadsA + i) * 1024 : BM * kBK + (wave * kLoadsB + i - kLoadsA) * 1024));
      p[i] += KG * kBK;
    }
  };

  constexpr int kMB = 2 * TM, kNB = 2 * TN;  // blocks of 16 rows and columns
  f32x4 acc[kMB][kNB];
#pragma unroll
  for (int i = 0; i < kMB; ++i)
#pragma unroll
    for (int j = 0; j < kNB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  struct Rows {
    Codes v;
    f32x4 s;
  };
  struct Cols {
    Codes v[kNB];
    float s;
  };
  // what this lane reads of a buffer: its places in the wave's first row and column, the two pieces
  // apart, and its rows' scales
  typedef __attribute__((address_space(3))) const uint8_t l_u8;
  typedef __attribute__((address_space(3))) const f8i4 l_f8i4;
  const int at_lo = l16 * kBK + ((quarter ^ swizzle(l16)) << 4), at_hi = l16 * kBK + (((4 + quarter) ^ swizzle(l16)) << 4);
  const int row0 = wm * 32 * TM * kBK, col0 = (BM + wn * 32 * TN) * kBK;
  l_u8* lds = (l_u8*)&sh[0][0];
  auto codes = [&](l_u8* lo, l_u8* hi, int block) {
    const f8i4 a = *(l_f8i4*)(lo + block * 16 * kBK), b = *(l_f8i4*)(hi + block * 16 * kBK);
    return Codes{i32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}};
  };
  typedef __attribute__((address_space(3))) const float l_f32;
  typedef __attribute__((address_space(3))) const f32x4 l_f32x4;
  const int first = wm * 32 * TM + 4 * quarter;  // this lane's first row
  l_f32* row_scales = (l_f32*)&all_scales[group][0][0][first / kOwnRows * kOwn + first % kOwnRows];
  l_f32* col_scale = (l_f32*)&all_scales[group][0][0][wave * kOwn + kOwnRows];
  struct Reader {
    l_u8 *row_lo, *row_hi, *col_lo, *col_hi;
    int scales;  // the step's, in floats
  };
  auto reader = [&](int buf, int set, int step) {
    l_u8* b = lds + buf * (int)sizeof(sh[0]);
    return Reader{b + row0 + at_lo, b + row0 + at_hi, b + col0 + at_lo, b + col0 + at_hi, (set * kSteps + step) * kWaves * kOwn};
  };
  auto fetch_rows = [&](Rows& f, const Reader& from, int i) {
    f.v = codes(from.row_lo, from.row_hi, i);
    // 16 rows on: in the same wave's part or a whole number of them on
    constexpr int kPer = kOwnRows < 16 ? 16 / kOwnRows * kOwn : kOwn;
    const int next = kOwnRows <= 16 ? i * kPer : i * 16 / kOwnRows * kOwn + i * 16 % kOwnRows;
    f.s = *(l_f32x4*)(row_scales + from.scales + next);
  };
  auto fetch_cols = [&](Cols& f, const Reader& from, int part, int parts) {
#pragma unroll
    for (int j = 0; j < kNB; ++j)
      if (j >= kNB * part / parts && j < kNB * (part + 1) / parts) f.v[j] = codes(from.col_lo, from.col_hi, j);
    if (part == 0) f.s = col_scale[from.scales];
  };
  // A block of rows' products are under way while those of the block before are added.
  f32x4 part[2][kNB], scale[2];
#pragma unroll
  for (int j = 0; j < kNB; ++j) part[1][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  scale[1] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto products = [&](const Rows& r, const Op* c, float sw, int i) {
    const Op x = Make::of(r.v);
    const int before = (i + kMB - 1) % kMB;
#pragma unroll
    for (int j = 0; j < kNB; ++j) {
      part[i % 2][j] = block_product(x, c[j]);
      scale[i % 2][j] = r.s[j] * sw;
      if (kNB == 2) scale[i % 2][2 + j] = r.s[2 + j] * sw;
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[before][j][v] = fmaf(scale[before % 2][v], part[before % 2][j][v], acc[before][j][v]);
      asm volatile("" : "+v"(acc[before][j]));  // formed here: put off to the step's end, sums kept every product in registers
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  static_assert(RING > 1 && RING <= kSteps, "a buffer is filled while another is read; the scales' sets are two");
  Rows rows[kMB];
  Cols c0, c1;
  int buf = 0, set = 0;
  Reader from = reader(0, 0, 0);
  // step S of kSteps; one RING steps on is loaded in it
  auto step = [&](auto number, const Cols& now, Cols& next) {
    constexpr int S = decltype(number)::value;
    // of the steps S + 2 .. S + RING - 1, whose loads may be under way when the next one's are in, one
    // may have come with scales
    constexpr bool kScales = (S + RING - 1) / kSteps > (S + 1) / kSteps;
    Op c[kNB];
#pragma unroll
    for (int j = 0; j < kNB; ++j) c[j] = Make::of(now.v[j]);
    // reads follow the products of what was read before: the compiler waits for all reads at once
    constexpr int kMeet = kMB / 2 - 1, kParts = kMB - kMeet;  // in which slot; those from it on
    int done = 0;
#pragma unroll
    for (int i = 0; i < kMB; ++i) {
      __builtin_amdgcn_sched_barrier(0);
      if (i == kMeet) {
        done = buf;
        buf = buf + 1 == RING ? 0 : buf + 1;
        meet_with_loads_but<(RING - 2) * kLoads + (kScales ? kSteps : 0)>();  // the next buffer is in
        from = reader(buf, S == kSteps - 1 ? set ^ 1 : set, (S + 1) % kSteps);
      }
      products(rows[i], c, now.s, i);
      if (i < kMeet) continue;
      if (i == kMeet)
#pragma unroll
        for (int k = 0; k < kMeet; ++k) fetch_rows(rows[k], from, k);
      fetch_rows(rows[i], from, i);
      if (i - kMeet < 2) fetch_cols(next, from, i - kMeet, 2);
      if (i == kMeet && S + RING == kSteps) stage_scales(set ^ 1);
      stage(done, i - kMeet, kParts);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  stage_scales(0);
#pragma unroll
  for (int r = 0; r < RING; ++r) {
    stage(r, 0, 1);
  }
  meet_with_loads_but<(RING - 1) * kLoads>();
#pragma unroll
  for (int i = 0; i < kMB; ++i) fetch_rows(rows[i], from, i);
  fetch_cols(c0, from, 0, 1);
  for (int left = (blocks - 1) / KG + 1;;) {  // two sets of columns in turn, so that each has its registers
    step(std::integral_constant<int, 0>(), c0, c1);
    if (--left == 0) break;
    step(std::integral_constant<int, 1>(), c1, c0);
    if (--left == 0) break;
    step(std::integral_constant<int, 2>(), c0, c1);
    if (--left == 0) break;
    step(std::integral_constant<int, 3>(), c1, c0);
    if (--left == 0) break;
    set ^= 1;
  }
#pragma unroll
  for (int j = 0; j < kNB; ++j)
#pragma unroll
    for (int v = 0; v < 4; ++v) acc[kMB - 1][j][v] = fmaf(scale[1][v], part[1][j][v], acc[kMB - 1][j][v]);

  // Each wave turns its sums in LDS, a block of 32 rows at a time (rows 16 bytes longer, so that
  // the four rows of a write use different banks), and reads four neighbouring channels of a
  // row a lane: whole lines are read and written from there on.
  meet_with_loads_but<0>();
  constexpr int kCols = 32 * TN, kRow = kCols + 4, kLanes = kCols / 4, kRows = 64 / kLanes;  // lanes of a row, rows a pass
  constexpr int kTurn = 32 * kRow;  // floats of a wave's block
  static_assert(sizeof(all) >= KG * kWaves * kTurn * 4, "the waves' blocks fit the buffers");
  float* turns = reinterpret_cast<float*>(&all[0][0][0]);
  float* turn = turns + wave_id * kTurn;
  const int c = lane % kLanes * 4, n = n0 + wn * kCols + c;
  float bias[4] = {0.f, 0.f, 0.f, 0.f};
  if (a.o.bias) load4(a.o.bias + n, a.N - n, bias);
  const bool whole = n0 + BN <= a.N;  // every channel of the tile is one
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int j = 0; j < kNB; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v) turn[(16 * b + 4 * quarter + v) * kRow + 16 * j + l16] = acc[2 * i + b][j][v];
    if (KG > 1) __syncthreads();
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    // each group stores a part of the rows, as long as there are any
    constexpr int kPasses = 32 / kRows >= KG ? 32 / kRows / KG : 1;
    const int rb = group * kPasses * kRows + lane / kLanes;
    const bool stores = group * kPasses * kRows < 32;
    const int row = (wm * TM + i) * 32 + rb;  // this lane's first row in the tile
    const float* from = turns + wave * kTurn + rb * kRow + c;
    if (!stores) {
    } else if (whole && m0 + (wm * TM + i + 1) * 32 <= a.T)
      store_rows<BF16, kPasses, kRows, kRow, KG, kWaves * kTurn, true>(a, m0 + row, n, from, bias);
    else
      store_rows<BF16, kPasses, kRows, kRow, KG, kWaves * kTurn, false>(a, m0 + row, n, from, bias);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (KG > 1 && i + 1 < TM) __syncthreads();
  }
}

}  // namespace

// The tiles, and what a block of K costs a CU in each (us), measured on bf16 products of 17 to 2048 tokens
// with 1001 to 7168 channels and K = 2048 to 7168. A large tile reads the fewest bytes per product, but
// too few of them leave CUs idle: the tile whose rounds over the 256 CUs cost least is taken. Against
// the next best tile that gives, at K = 7168 in a loop over one set of buffers: 2048 x 7168 121 us
// (128 x 128: 160), 1024 x 7168 60 (128 x 128: 80), 512 x 7168 38 (64 x 128: 51), 256 x 7168 25.5 (64 x 64:
// 31), 128 x 7168 17.0 (64 x 128: 24.6), 64 x 7168 14.6 (64 x 64: 16.8), 16 x 7168 11.9 (64 x 32: 12.9).
// fp32 products cost more a block, in the same proportions: 2048 x 7168 253 us (64 x 128: 284), 1024 x
// 7168 127 (156), 512 x 7168 65 (64 x 128: 81), 256 x 7168 43 (64 x 64: 45), 128 x 7168 24 (64 x 32: 30), 64 x
// 7168 16.6 (32 x 32: 22), 16 x 7168 12.8 (64 x 32: 16.3). Over these and 1001 x 2064, 2048 x 2048, 4096 x
// 7168 and 5120 x 4096 channels x K, 16 to 2048 tokens, no tile beats the chosen one by 2% in either type.
constexpr Tile kTiles[] = {{128, 256, 0.93f}, {128, 128, 0.66f}, {64, 128, 0.43f}, {64, 64, 0.29f}, {64, 32, 0.235f}, {32, 32, 0.18f}};

template <bool BF16, int WM, int WN, int TM, int TN, int RING, int KG>
static void gemm_tile(const Fp8Args& a, hipStream_t s) {
  const int mt = (a.T - 1) / (32 * TM * WM) + 1, nt = (a.N - 1) / (32 * TN * WN) + 1;
  hipLaunchKernelGGL((k_fp8_gemm<WM, WN, TM, TN, RING, KG, BF16>), dim3(mt * nt), dim3(64 * WM * WN * KG), 0, s, a, mt);
}

template <bool BF16>
static void gemm(const Fp8Args& a, hipStream_t s) {
  switch (choose_tile(kTiles, a.T, a.N, BF16 ? 0 : 1)) {
    case 0:
      if constexpr (BF16) return gemm_tile<BF16, 2, 4, 2, 2, 3, 1>(a, s);
    case 1: return gemm_tile<BF16, 2, 4, 2, 1, 4, 1>(a, s);
    case 2: return gemm_tile<BF16, 2, 4, 1, 1, 4, 1>(a, s);
    case 3: return gemm_tile<BF16, 2, 2, 1, 1, 4, 2>(a, s);
    case 4: return gemm_tile<BF16, 2, 1, 1, 1, 3, 4>(a, s);
    default: return gemm_tile<BF16, 1, 1, 1, 1, 4, 4>(a, s);
  }
}

void launch_fp8_gemm(const Fp8Args& a, bool out_bf16, hipStream_t s) {
  if (out_bf16)
    gemm<true>(a, s);
  else
    gemm<false>(a, s);
}

}  // namespace moe
