// 8-bit matrix product for many rows, and its gated form: tiles of tokens x channels on
// v_mfma_i32_16x16x64_i8.
//
// Lane layout of the 16x16x64 MFMA: lane l supplies 16 bytes of row l % 16 of each operand at
// K offset 16 (l / 16), and receives the sums of column l % 16 and rows 4 (l / 16) .. + 3.
// Tokens are the row operand and channels the column operand. (On random codes the matrix
// pipes are held by power: 256 CUs of this instruction alone run at 2.1 GHz and 4.2 POPS, of
// 32x32x32 at 1.75 GHz and 3.7.)
//
// A tile of BM tokens x BN channels runs over K in steps of BK bytes (64 or 128) through a
// ring of LDS buffers, filled by loads that go from memory to LDS directly (16 bytes a lane,
// 1024 / BK rows an instruction). In LDS the 16-byte pieces of row r stand at places
// piece ^ swizzle(r): an instruction writes its lanes' bytes in lane order, so each lane
// fetches the piece that belongs at its place, and the lanes that a read serves at once use
// every bank once. Pieces past K come from a line of zeros.
//
// A step is two halves: of 64 bytes of K each where a step has 128, else of half of the rows
// each. The operands of one are read from LDS while the products of the other run; the
// barrier that frees the oldest buffer and opens the next stands between the two, so that
// it, too, is covered by products.
//
// What bounds it: 2048 x 7168 x 7168 takes 97 us (2.17 POPS) in a loop over one set of
// buffers, 103 us with inputs and outputs all from HBM. A 64-byte step of the 256 x 256 tile is
// 1088 cycles of its MFMAs and runs in about 1390, at the 1.8 GHz that the power limit
// leaves; without the loads the same loop takes 73 us, and on loads that all hit L2 98% of
// its time, so it is their way into LDS beside the products that costs, not memory. The
// rest, about 10 us, is the launch, the first loads and the epilogue's bytes.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "int8_out.h"
#include "tiles.h"

namespace moe {
namespace {

// Place of row r's piece p: p ^ swizzle(r). A 16-byte read serves sixteen lanes at once, lanes
// 0-3, 12-15, 20-23 and 24-27 of each half wave and then the others: of 64-byte rows those
// are the row quads 0 and 3 of one piece and 1 and 2 of the next, which -(quad) % 4 keeps in
// different banks (quad itself: every read took twice as long, 9.9 M conflict cycles in 2048
// x 7168 x 7168); of 128-byte rows r / 2 does.
template <int BK>
__device__ __forceinline__ int swizzle(int r) {
  return BK == 64 ? (-(r >> 2)) & 3 : (r >> 1) & 7;
}

// what pieces past K are read from
__device__ const i32x4 zero_piece = {0, 0, 0, 0};

// PASSES rows, ROWS apart, of four channels each, from their sums in LDS. WHOLE: every row
// and channel is one of the matrix's, and what the rows need is loaded for all of them
// before it is used. A sum is in PARTS parts, PART ints apart.
template <bool GATED, bool BF16, int PASSES, int ROWS, int LDROW, int PARTS, int PART, bool WHOLE>
__device__ __forceinline__ void store_rows(const Int8Args& a, int t0, int n, const float* sx, const int* from,
                                           const float* sw, const float* su, const float* bias) {
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
      i32x4 s = *reinterpret_cast<const i32x4*>(from + r * LDROW);
      for (int k = 1; k < PARTS; ++k) s += *reinterpret_cast<const i32x4*>(from + k * PART + r * LDROW);
      if (GATED) {
        i32x4 u = *reinterpret_cast<const i32x4*>(from + r * LDROW + 16);
        for (int k = 1; k < PARTS; ++k) u += *reinterpret_cast<const i32x4*>(from + k * PART + r * LDROW + 16);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[p][e] = gated_value(s[e], u[e], sx[r], sw[e], su[e]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[p][e] = int8_scaled(s[e], sx[r], sw[e], bias[e]);
      }
    }
    if (!GATED && a.o.y) {
#pragma unroll
      for (int p = 0; p < kAt; ++p)
        if (WHOLE || t0 + (p0 + p) * ROWS < a.T) load4(a.o.y + (t0 + (p0 + p) * ROWS) * a.o.ld_y + n, left, more[p]);
#pragma unroll
      for (int p = 0; p < kAt; ++p)
#pragma unroll
        for (int e = 0; e < 4; ++e) v[p][e] += more[p][e];
    }
    if (!GATED && a.o.res) {
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

// WM x WN waves, each 32 TM x 32 TN; RING buffers. KG such groups of waves take the steps of
// K in turn, each with buffers of its own, and add their sums at the end. GATED: of every 32
// channels of the tile the first 16 are gate rows and the others the same rows of up, and h
// is stored in fp32.
template <int WM, int WN, int TM, int TN, int BK, int RING, int KG, bool GATED, bool BF16>
__global__ __launch_bounds__(64 * WM* WN* KG) void k_int8_gemm(Int8Args a, int mtiles) {
  constexpr int kWaves = WM * WN, BM = 32 * TM * WM, BN = 32 * TN * WN;
  constexpr int kPieces = BK / 16, kRowsPer = 64 / kPieces;  // pieces of a row; rows of a load instruction
  constexpr int kLoadsA = BM / kRowsPer / kWaves, kLoadsB = BN / kRowsPer / kWaves;  // instructions of a wave per step
  static_assert(kLoadsA * kRowsPer * kWaves == BM && kLoadsB * kRowsPer * kWaves == BN, "rows divide among the waves");
  constexpr int kLoads = kLoadsA + kLoadsB;
  __shared__ __attribute__((aligned(1024))) uint8_t all[KG][RING][(BM + BN) * BK];
  const int lane = threadIdx.x & 63, wave_id = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = KG == 1 ? 0 : wave_id / kWaves, wave = KG == 1 ? wave_id : wave_id % kWaves;
  uint8_t(*sh)[(BM + BN) * BK] = all[group];
  const int tile = xcd_order(blockIdx.x, gridDim.x);
  const int m0 = tile % mtiles * BM, n0 = tile / mtiles * (GATED ? BN / 2 : BN);

  __shared__ float rows_sx[BM];
  for (int i = threadIdx.x; i < BM; i += 64 * kWaves * KG) rows_sx[i] = a.o.sx[min(m0 + i, a.T - 1)];
  // this lane's channels in the epilogue: columns c .. c + 3 of the wave's (gated: gate
  // columns; up's are 16 on), their scales and bias
  constexpr int kCols = 32 * TN, kRow = kCols + 4;
  constexpr int kLanes = kCols / 4 / (GATED ? 2 : 1), kRows = 64 / kLanes;  // lanes of a row, rows a pass
  const int wm = wave / WN, wn = wave % WN, l16 = lane & 15, quarter = lane >> 4;
  const int lc = lane % kLanes * 4, c = GATED ? lc / 16 * 32 + lc % 16 : lc;
  const int n = n0 + wn * (GATED ? kCols / 2 : kCols) + lc;
  float sw[4], su[4] = {0.f, 0.f, 0.f, 0.f}, bias[4] = {0.f, 0.f, 0.f, 0.f};
  load4(a.o.sw + n, a.N - n, sw);
  if (GATED) load4(a.o.sw + a.N + n, a.N - n, su);
  if (!GATED && a.o.bias) load4(a.o.bias + n, a.N - n, bias);

  // this lane's piece of each row that it fetches; rows past the last are read as the last,
  // and not stored
  const int lrow = lane / kPieces;
  const int8_t* p[kLoads];
  int at[kLoads];  // its offset in K
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const bool in_a = i < kLoadsA;
    const int r = (in_a ? wave * kLoadsA + i : wave * kLoadsB + i - kLoadsA) * kRowsPer + lrow;
    int64_t row = in_a ? min(m0 + r, a.T - 1) : min(n0 + r, a.N - 1);
    if (GATED && !in_a) row = (int64_t)min(n0 + r / 32 * 16 + r % 16, a.N - 1) + (r & 16 ? a.N : 0);
    at[i] = ((lane % kPieces) ^ swizzle<BK>(r)) * 16;
    p[i] = (in_a ? a.x + row * a.ld_x : a.w + row * a.ld_w) + group * BK + at[i];
  }
  const int8_t* zeros = reinterpret_cast<const int8_t*>(&zero_piece);
  const uint32_t ring = (uint32_t)(uintptr_t)(lvoid*)&sh[0][0];
  int kat = group * BK;  // K offset of the next step to load
  // the part'th of `parts` parts of the next step's pieces into buffer `buf` (past the last
  // step: zeros)
  auto stage = [&](int buf, int part, int parts) {
    if (part == 0) {
      if (kat + BK > a.K) {  // the last of K is in it, or nothing
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
          if (kat + at[i] >= a.K) p[i] = zeros;
      }
      kat += KG * BK;
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      if (i < kLoads * part / parts || i >= kLoads * (part + 1) / parts) continue;
      const int to = i < kLoadsA ? (wave * kLoadsA + i) * 1024 : BM * BK + (wave * kLoadsB + i - kLoadsA) * 1024;
      load_to_lds(p[i], ring + buf * (BM + BN) * BK + to);
      p[i] += KG * BK;
    }
  };

  // blocks of 16 rows and columns of the wave, and the row blocks of a half
  constexpr int kMB = 2 * TM, kNB = 2 * TN, kHalfMB = BK == 128 ? kMB : kMB / 2;
  i32x4 acc[kMB][kNB];
#pragma unroll
  for (int i = 0; i < kMB; ++i)
#pragma unroll
    for (int j = 0; j < kNB; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
  struct Rows {
    i32x4 v[kHalfMB];
  };
  struct Cols {
    i32x4 v[kNB];
  };
  // the part'th of `parts` parts of a half's rows, and of its columns
  auto fetch_rows = [&](Rows& f, int buf, int h, int part, int parts) {
    const int r0 = wm * 32 * TM + (BK == 128 ? 0 : h * kHalfMB * 16);
    const int off = l16 * BK + ((((BK == 128 ? 4 * h : 0) + quarter) ^ swizzle<BK>(l16)) << 4);
#pragma unroll
    for (int i = 0; i < kHalfMB; ++i)
      if (i >= kHalfMB * part / parts && i < kHalfMB * (part + 1) / parts)
        f.v[i] = *reinterpret_cast<const i32x4*>(&sh[buf][(r0 + 16 * i) * BK + off]);
  };
  auto fetch_cols = [&](Cols& f, int buf, int h, int part, int parts) {
    const int off = l16 * BK + ((((BK == 128 ? 4 * h : 0) + quarter) ^ swizzle<BK>(l16)) << 4);
#pragma unroll
    for (int j = 0; j < kNB; ++j)
      if (j >= kNB * part / parts && j < kNB * (part + 1) / parts)
        f.v[j] = *reinterpret_cast<const i32x4*>(&sh[buf][(BM + wn * 32 * TN + 16 * j) * BK + off]);
  };
  auto products = [&](const Rows& r, const Cols& c, int h, int i) {
    const int at_row = BK == 128 ? i : h * kHalfMB + i;
#pragma unroll
    for (int j = 0; j < kNB; ++j) acc[at_row][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(r.v[i], c.v[j], acc[at_row][j], 0, 0, 0);
  };
  // A half has kHalfMB slots of kNB products; the operands of the next are asked for in the
  // first of them, so that they are in when its products start, and loads follow.
  // A freed buffer is filled in this half and the next (at once, 128 x 256 tiles on 112 CUs
  // take 43 us for 39, on 256 CUs 58 for 56.5), for which the ring has to hold another.
  static_assert(RING > 2, "the next step's buffer is full before the freed one is");
  constexpr int kReadSlots = kHalfMB / 2, kParts = kHalfMB - kReadSlots, kAllParts = 2 * kParts;
  Rows r0, r1;
  Cols c0, c1;
  int buf = 0, fill = RING - 1;
  // One step: rows r0 and columns `now` are in registers at its start, those of the next
  // step's first half at its end (columns in `next`, which with BK = 128 holds the second
  // half's in between).
  auto step = [&](Cols& now, Cols& next) {
#pragma unroll
    for (int i = 0; i < kHalfMB; ++i) {
      __builtin_amdgcn_sched_barrier(0);
      products(r0, now, 0, i);
      __builtin_amdgcn_sched_barrier(0);
      if (i < kReadSlots) {
        if (BK == 128) fetch_cols(next, buf, 1, i, kReadSlots);
        fetch_rows(r1, buf, 1, i, kReadSlots);
      }
      if (i >= kReadSlots) stage(fill, kParts + i - kReadSlots, kAllParts);
    }
    __builtin_amdgcn_sched_barrier(0);
    const int done = buf;  // every wave has all of it in registers at the barrier
    buf = buf + 1 == RING ? 0 : buf + 1;
    meet_with_loads_but<(RING - 2) * kLoads>();  // the next buffer is in, this one's operands too
#pragma unroll
    for (int i = 0; i < kHalfMB; ++i) {
      __builtin_amdgcn_sched_barrier(0);
      products(r1, BK == 128 ? next : now, 1, i);
      __builtin_amdgcn_sched_barrier(0);
      if (i < kReadSlots) {
        fetch_cols(BK == 128 ? now : next, buf, 0, i, kReadSlots);
        fetch_rows(r0, buf, 0, i, kReadSlots);
      }
      if (i >= kReadSlots) stage(done, i - kReadSlots, kAllParts);
    }
    fill = done;
  };
#pragma unroll
  for (int r = 0; r < RING - 1; ++r) stage(r, 0, 1);
#pragma unroll
  for (int q = 0; q < kParts; ++q) stage(RING - 1, q, kAllParts);
  meet_with_loads_but<(RING - 2) * kLoads + kLoads / 2>();
  fetch_rows(r0, 0, 0, 0, 1);
  fetch_cols(c0, 0, 0, 0, 1);
  if (BK == 128) {
    for (int k = 0; k < a.K; k += KG * BK) step(c0, c1);
  } else {  // two steps a turn, so that each set of columns has its registers; the second may be zeros
    for (int k = 0; k < a.K; k += 2 * KG * BK) {
      step(c0, c1);
      step(c1, c0);
    }
  }

  // Each wave turns its sums in LDS, a block of 32 rows at a time (rows 16 bytes longer, so
  // that the four rows of a write use different banks), and reads four neighbouring
  // channels of a row a lane: whole lines are read and written from there on.
  meet_with_loads_but<0>();
  constexpr int kTurn = 32 * kRow;  // ints of a wave's block
  static_assert(sizeof(all) >= KG * kWaves * kTurn * 4, "the waves' blocks fit the buffers");
  int* blocks = reinterpret_cast<int*>(&all[0][0][0]);
  int* turn = blocks + wave_id * kTurn;
  const bool whole = n0 + (GATED ? BN / 2 : BN) <= a.N;  // every channel of the tile is one
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
    const int r0 = (wm * TM + i) * 32 + rb;  // this lane's first row in the tile
    const int* from = blocks + wave * kTurn + rb * kRow + c;
    if (!stores) {
    } else if (whole && m0 + (wm * TM + i + 1) * 32 <= a.T)
      store_rows<GATED, BF16, kPasses, kRows, kRow, KG, kWaves * kTurn, true>(a, m0 + r0, n, rows_sx + r0, from, sw, su, bias);
    else
      store_rows<GATED, BF16, kPasses, kRows, kRow, KG, kWaves * kTurn, false>(a, m0 + r0, n, rows_sx + r0, from, sw, su, bias);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (KG > 1 && i + 1 < TM) __syncthreads();
  }
}

}  // namespace

// The tiles, and what 128 bytes of K cost a CU in each (us), measured on products of 64 to
// 2048 tokens with 2048 to 7168 channels and K. A large tile reads the fewest bytes per
// product, but too few of them leave CUs idle: the tile whose rounds over the 256 CUs cost
// least is taken. Against the next best tile that gives, at K = 7168, in a loop over one set
// of buffers: 2048 x 7168 97 us (128 x 256: 99), 2048 x 4096 59 (128 x 128: 66), 1024 x 7168
// 54 (128 x 128: 59), 512 x 7168 33 (64 x 128: 39), 300 x 7168 28 (64 x 128: 36), 256 x 7168
// 21 (64 x 64: 26), 128 x 7168 14.8 (64 x 128: 18.4), 64 x 7168 12.5 (64 x 64: 13.7). The
// smaller tiles are short of products to cover a step's LDS reads and barrier, so that two or
// four groups of waves take the steps in turn (64 x 64 in one group: 18.3 us for 128 x 7168;
// 64 x 32 11.3 and 64 x 64 13.2 us for 128 x 4096; 32 x 32 8.4, 64 x 32 9.1 and 64 x 64 11.1
// us for 64 x 4096). 257 to 384 tokens run as 384 rows, on 160 to 168 CUs of the larger shapes.
constexpr Tile kTiles[] = {{256, 256, 1.65f}, {128, 256, 0.88f}, {128, 128, 0.53f}, {64, 128, 0.35f},
                          {64, 64, 0.25f},   {64, 32, 0.20f},   {32, 32, 0.16f}};

template <bool GATED, bool BF16, int WM, int WN, int TM, int TN, int BK, int RING, int KG>
static void gemm_tile(const Int8Args& a, hipStream_t s) {
  const int mt = (a.T - 1) / (32 * TM * WM) + 1, nt = (a.N - 1) / (32 * TN * WN / (GATED ? 2 : 1)) + 1;
  hipLaunchKernelGGL((k_int8_gemm<WM, WN, TM, TN, BK, RING, KG, GATED, BF16>), dim3(mt * nt), dim3(64 * WM * WN * KG), 0, s, a, mt);
}

template <bool GATED, bool BF16>
static void gemm(const Int8Args& a, hipStream_t s) {
  switch (choose_tile(kTiles, a.T, GATED ? 2 * (int64_t)a.N : a.N)) {
    case 0: return gemm_tile<GATED, BF16, 2, 4, 4, 2, 64, 4, 1>(a, s);
    case 1: return gemm_tile<GATED, BF16, 2, 4, 2, 2, 128, 3, 1>(a, s);
    case 2: return gemm_tile<GATED, BF16, 2, 4, 2, 1, 128, 4, 1>(a, s);
    case 3: return gemm_tile<GATED, BF16, 2, 4, 1, 1, 128, 4, 1>(a, s);
    case 4: return gemm_tile<GATED, BF16, 2, 2, 1, 1, 128, 4, 2>(a, s);
    case 5: return gemm_tile<GATED, BF16, 2, 1, 1, 1, 128, 3, 4>(a, s);
    default: return gemm_tile<GATED, BF16, 1, 1, 1, 1, 128, 4, 4>(a, s);
  }
}

void launch_int8_gemm(const Int8Args& a, bool out_bf16, hipStream_t s) {
  if (out_bf16)
    gemm<false, true>(a, s);
  else
    gemm<false, false>(a, s);
}

void launch_int8_gated_gemm(const Int8Args& a, hipStream_t s) { gemm<true, false>(a, s); }

}  // namespace moe
