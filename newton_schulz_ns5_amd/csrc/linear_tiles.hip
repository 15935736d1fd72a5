// The linear product and its gradients as tiled MFMA products on gfx950.
//
// C = A B^T with either operand stored K-contiguous ("row") or with its own
// index contiguous ("col"); see LinGemm.  The work is 2 M N K operations on
// operands that are each re-read once per tile of the other, so it is bound by
// the matrix units once a tile is large enough; the kernel is built to keep
// them fed:
//  - one workgroup per BM x BN output tile, its waves in WM x WN, each wave a
//    block of 16 x 16 products (v_mfma_f32_16x16x32_bf16: 3 % faster here than
//    the 32x32x16 form, which moves more accumulator values per operation;
//    fp32: 16x16x4).  256 x 256: eight waves of 128 x 64, two per SIMD;
//    256 x 128: eight of 64 x 64; 128 and 64: four waves, two and three or four
//    workgroups per CU, for outputs with too few large tiles to fill the chip;
//  - K advances by 128 bytes of a row (64 bf16 or 32 fp32 values) per slice,
//    brought HBM -> LDS directly into a ring of operand slots, one and a half
//    to two slices ahead, with one barrier per slice; loads, fragment reads
//    and MFMAs are interleaved in fixed slots;
//  - row operands: a slot row is 128 bytes of K with its 16-byte chunks
//    XOR-swizzled by (row / 2) mod 8, one ds_read_b128 per fragment; col
//    operands: a slot row is one K value of all the tile's indices, read
//    through the transposing ds_read_b64_tr_b16 (bf16) or single words (fp32),
//    with its blocks XOR-swizzled so that no bank is read twice;
//  - every LDS address of a lane is one register per operand plus constants: a
//    version that formed them per read spilled six registers in the product
//    of two col operands, whose reloads waited out the loads in flight
//    (14336 x 4096 over 4096 in 256 x 256 tiles: 537 us where this takes 400 to
//    433, by the box's clock).
// What bounds it: 4096 x 4096 over 14336 runs at 1337 TFLOP/s (the library's
// product at 1263 on the same box) with the matrix units about 70 % busy, at a
// clock that power holds near 1.65 GHz; the epilogue and the pipeline's start
// cost about 8 us per round of workgroups.
// Ragged sizes cost nothing in the loop: rows past the end repeat the last one
// (their products are not stored), K values past the end are zeros from the
// buffer descriptor's bounds check (which the loads of the last slice are sent
// past), for both operands, so nothing of a neighbouring buffer enters a sum.
#include "layer_internal.h"
#include "linear_epilogue.h"

#include <algorithm>

namespace muon {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

#define MUON_LDS(p) ((__attribute__((address_space(3))) void*)(p))

constexpr int ROWB = 128;   // bytes of K per slice
constexpr int kOut = (int)0x80000000;  // a byte offset past every descriptor's end

// Workgroup -> (split, tile row, tile column): XCD x takes 32 consecutive
// tiles of every 8 x 32, tiles run in bands of four rows, so the tiles an XCD
// works on together share their operand panels in its L2.
__device__ __forceinline__ void decode(int tiles_m, int tiles_n, int& sp, int& tm, int& tn) {
  constexpr int CH = 32, GM = 4;
  const int G = gridDim.x, wg = blockIdx.x, x = wg & 7, k = wg >> 3;
  const int full = (G / (8 * CH)) * (8 * CH);
  const int pid = wg < full ? (k / CH) * (8 * CH) + x * CH + (k % CH) : wg;
  const int tiles = tiles_m * tiles_n;
  sp = pid / tiles;
  const int t = pid - sp * tiles;
  const int span = GM * tiles_n, grp = t / span, first = grp * GM;
  const int gsz = min(tiles_m - first, GM);
  const int r = t - grp * span;
  tm = first + r % gsz;
  tn = r / gsz;
}

// LDS reads and addresses of one operand: EXT its tile edge, COL its layout.
template <typename T, int EXT, bool COL>
struct Operand {
  static constexpr bool BF = sizeof(T) == 2;
  static constexpr int ES = sizeof(T);
  static constexpr int KS = ROWB / ES;
  static constexpr int BYTES = EXT * ROWB;    // of one slot
  static constexpr int CROWB = EXT * ES;      // col: bytes of one K row
  static constexpr int CCH = CROWB / 16;      // col: 16-byte chunks of it
  // XOR key of a K row of a col slot.  bf16, on 32-byte blocks: 32 lanes of a
  // transposing read touch one block of the rows 8 g + 0 .. 3 of two
  // neighbouring g (and, in a 128-byte row, rows of equal parity share banks).
  // fp32, on 64-byte blocks: a word read touches one block of rows 4 g of four
  // g.
  static __device__ __forceinline__ int key(int row) {
    if constexpr (!BF) return (row >> 2) & 3;
    else if constexpr (EXT == 64) return ((row >> 1) & 1) | (((row >> 3) & 1) << 1);
    else return (row & 3) | (((row >> 3) & 1) << 2);
  }
  // Global chunk that the load landing at (slot row, chunk c) fetches.
  static __device__ __forceinline__ int source_chunk(int row, int c) {
    if constexpr (!COL) return c ^ ((row >> 1) & 7);
    else if constexpr (BF) return 2 * ((c >> 1) ^ key(row)) + (c & 1);
    else return 4 * ((c >> 2) ^ key(row)) + (c & 3);
  }
  // A lane's address within a slot for its wave's indices from `at` on (a
  // multiple of the wave's extent): see read().
  static __device__ __forceinline__ uint32_t lane_base(int lane, int at) {
    const int i = lane & 15, g = lane >> 4;
    if constexpr (!COL) return (uint32_t)((at + i) * ROWB + (g ^ ((i >> 1) & 7)) * 16);
    else if constexpr (BF) return (uint32_t)((8 * g + (i >> 2)) * CROWB + ((at >> 4) ^ key(8 * g + (i >> 2))) * 32 + (i & 3) * 8);
    else return (uint32_t)(4 * g * CROWB + ((at >> 4) ^ key(4 * g)) * 64 + i * 4);
  }
  // Fragment f of half hf of a slice: for index 16 f + l % 16 of the wave's,
  // 16 bytes of K: bf16, values 32 hf + 8 g .. + 7 (g = l / 16), one product;
  // fp32, values 16 hf + 4 g .. + 3, one for each of four products.
  static __device__ __forceinline__ u32x4 read(uint32_t base, int hf, int f) {
    typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    typedef __attribute__((address_space(3))) uint32_t lds_u32;
    if constexpr (!COL) {
      return *(const lds_u32x4*)(uintptr_t)((base ^ (uint32_t)(hf * 64)) + (uint32_t)(f * 16 * ROWB));
    } else if constexpr (BF) {
      const uint32_t at = (base ^ (uint32_t)(f * 32)) + (uint32_t)(hf * 32 * CROWB);
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(uintptr_t)at);
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(uintptr_t)(at + 4 * CROWB));
      return __builtin_bit_cast(u32x4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      const uint32_t at = (base ^ (uint32_t)(f * 64)) + (uint32_t)(hf * 16 * CROWB);
      u32x4 v;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = *(const lds_u32*)(uintptr_t)(at + e * CROWB);
      return v;
    }
  }
};

template <typename T, int KIND, int BM, int BN, int WM, int WN, int DEPTH>
__global__ __launch_bounds__(WM * WN * 64, 1) void linear_tile_kernel(const LinGemm p) {
  constexpr bool BF = sizeof(T) == 2;
  constexpr bool ACOL = KIND == kColCol, BCOL = KIND != kRowRow;
  typedef Operand<T, BM, ACOL> OA;
  typedef Operand<T, BN, BCOL> OB;
  constexpr int ES = sizeof(T), KS = ROWB / ES;
  constexpr int NW = WM * WN, NTH = NW * 64;
  constexpr int WT = BM / WM, WC = BN / WN;      // wave tile
  constexpr int F = WT / 16, FN = WC / 16, FH = F / 2;
  constexpr int DPA = BM / NW / 8, DPB = BN / NW / 8;  // load instructions per wave, operand and slice
  // Ring: DEPTH slots of each operand, or (DEPTH 0) five that both share: A of
  // slice t in 2 t mod 5, B in 2 t + 1 mod 5.
  constexpr bool RING5 = DEPTH == 0;
  constexpr int RING_A = RING5 ? 5 * OA::BYTES : DEPTH * OA::BYTES;
  constexpr int RING = RING5 ? RING_A : RING_A + DEPTH * OB::BYTES;
  constexpr int RH = BM / 2, PITCH = BN + 4;
  constexpr int LDS_BYTES = RING > RH * PITCH * 4 ? RING : RH * PITCH * 4;
  static_assert(DPA >= 1 && DPB >= 1 && (!RING5 || (DPB % 2 == 0 && BM == BN)) && (RING5 || DEPTH >= 3) && F % 2 == 0 && FN % 2 == 0, "tile shape");
  static_assert((WT & (WT - 1)) == 0 && (WC & (WC - 1)) == 0, "fragment indices are XORed into addresses");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[LDS_BYTES];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int tiles_m = (int)((p.M + BM - 1) / BM), tiles_n = (int)((p.N + BN - 1) / BN);
  int sp, tm, tn;
  decode(tiles_m, tiles_n, sp, tm, tn);
  const int64_t i0 = (int64_t)tm * BM, j0 = (int64_t)tn * BN;

  // This workgroup's slices of K: chunk sp of the split sum.
  const int slices = (int)((p.K + KS - 1) / KS);
  const int t0 = p.split > 1 ? (int)((int64_t)sp * slices / p.split) : 0;
  const int t1 = p.split > 1 ? (int)((int64_t)(sp + 1) * slices / p.split) : slices;
  const int KT = __builtin_amdgcn_readfirstlane(t1 > t0 ? t1 - t0 : 1);  // an empty sum is one slice of zeros
  const int64_t kbeg = (int64_t)t0 * KS;
  const int64_t kend = (int64_t)t1 * KS < p.K ? (int64_t)t1 * KS : p.K;
  const int Kc = (int)(kend - kbeg);                // K values of this workgroup

  // Each lane's byte offset for each load instruction.  Instruction q of a
  // wave fills the 1024 bytes of a slot from (wave DP + q) 1024 on, lane l its
  // 16 bytes there: slot row and chunk follow.
  int avo[DPA], bvo[DPB];
  const int64_t arows = p.M - i0, brows = p.N - j0;
  const int lda = __builtin_amdgcn_readfirstlane((int)p.lda), ldb = __builtin_amdgcn_readfirstlane((int)p.ldb);
  auto offset = [&](auto op, bool col, int at, int ld, int64_t rows) {
    typedef decltype(op) O;
    if (col) {
      const int row = at / O::CROWB, c = (at % O::CROWB) / 16;
      return row * ld * ES + O::source_chunk(row, c) * 16;
    }
    const int row = at / ROWB, c = (at % ROWB) / 16;
    return (row < rows ? row : (int)rows - 1) * ld * ES + O::source_chunk(row, c) * 16;
  };
#pragma unroll
  for (int q = 0; q < DPA; ++q) avo[q] = offset(OA{}, ACOL, (wave * DPA + q) * 1024 + lane * 16, lda, arows);
#pragma unroll
  for (int q = 0; q < DPB; ++q) bvo[q] = offset(OB{}, BCOL, (wave * DPB + q) * 1024 + lane * 16, ldb, brows);
  // The last slice's loads: row chunks past K go past the descriptor's end.
  const int klast = Kc - (KT - 1) * KS;             // K values of the last slice (0: none)
  auto tail = [&](int vo, int at) {
    const int row = at / ROWB, c = (at % ROWB) / 16;
    return (c ^ ((row >> 1) & 7)) * (16 / ES) < klast ? vo : kOut;
  };
  // A row operand's panel: its descriptor spans the tile's rows from K value
  // kbeg on.  A col operand's: rebased every slice, ending after its last K
  // row's columns (rounded up to whole chunks).
  const char* const Ab = (const char*)p.A + (ACOL ? kbeg * p.lda + i0 : i0 * p.lda + kbeg) * ES;
  const char* const Bb = (const char*)p.B + (BCOL ? kbeg * p.ldb + j0 : j0 * p.ldb + kbeg) * ES;
  auto span = [&](int64_t rows, int ext, int64_t ld) {
    const int64_t r = rows < ext ? rows : ext;
    return Kc > 0 ? ((r - 1) * ld + (Kc + 16 / ES - 1) / (16 / ES) * (16 / ES)) * ES : 0;
  };
  const i32x4 ars = rsrc_words(Ab, ACOL ? 0 : span(arows, BM, p.lda));
  const i32x4 brs = rsrc_words(Bb, BCOL ? 0 : span(brows, BN, p.ldb));
  // Scalar arithmetic only (32-bit compares and products of values made uniform
  // once), so that the words stay in scalar registers.
  auto uni = [](int v) { return (int)__builtin_amdgcn_readfirstlane(v); };
  auto uni64 = [&](const char* v) {
    return (uint64_t)(uint32_t)uni((int)(uint32_t)(uint64_t)v) | ((uint64_t)(uint32_t)uni((int)((uint64_t)v >> 32)) << 32);
  };
  const uint64_t Au = uni64(Ab), Bu = uni64(Bb);
  const int kcol = (int)((p.Kcol < kend ? p.Kcol : kend) - kbeg);
  auto col_bytes = [&](int ld, int64_t rows, int ext, int left) {
    const int cols = rows < ext ? ((int)rows + 16 / ES - 1) / (16 / ES) * (16 / ES) : ext;
    return left <= 0 ? 0 : (((left < KS ? left : KS) - 1) * ld + cols) * ES;
  };
  const int left = kcol - (KT - 1) * KS;
  const int afull = uni(ACOL ? col_bytes(lda, arows, BM, KS) : 0), alast = uni(ACOL ? col_bytes(lda, arows, BM, left) : 0);
  const int bfull = uni(BCOL ? col_bytes(ldb, brows, BN, KS) : 0), blast = uni(BCOL ? col_bytes(ldb, brows, BN, left) : 0);
  auto col_rsrc = [&](uint64_t base, int ld, int full, int end, int t) {
    const uint64_t a = base + (uint64_t)(uint32_t)t * (uint32_t)(KS * ld * ES);
    i32x4 r;
    r[0] = (int)(uint32_t)a;
    r[1] = (int)((uint32_t)(a >> 32) & 0xffffu);
    r[2] = t >= KT - 1 ? end : full;
    r[3] = 0x00020000;
    return r;
  };

  const uint32_t smem_lds =
      __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)smem);
  // Load instruction q of an operand of slice t into the slot at `slot`.
  // Slices past the last (the pipeline runs ahead) repeat it into slots nobody
  // reads.
  auto load_a = [&](int t, uint32_t slot, int q) {
    const bool last = t >= KT - 1;
    const int tc = last ? KT - 1 : t, at = (wave * DPA + q) * 1024;
    if constexpr (ACOL) lds_dma16_asm(col_rsrc(Au, lda, afull, alast, tc), slot + at, avo[q], 0);
    else lds_dma16_asm(ars, slot + at, last ? tail(avo[q], at + lane * 16) : avo[q], tc * ROWB);
  };
  auto load_b = [&](int t, uint32_t slot, int q) {
    const bool last = t >= KT - 1;
    const int tc = last ? KT - 1 : t, at = (wave * DPB + q) * 1024;
    if constexpr (BCOL) lds_dma16_asm(col_rsrc(Bu, ldb, bfull, blast, tc), slot + at, bvo[q], 0);
    else lds_dma16_asm(brs, slot + at, last ? tail(bvo[q], at + lane * 16) : bvo[q], tc * ROWB);
  };
  // Slot of the next slice of the same operand.
  auto next_a = [&](uint32_t s) {
    const uint32_t step = RING5 ? 2 * OA::BYTES : OA::BYTES, end = smem_lds + RING_A;
    return s + step >= end ? s + step - RING_A : s + step;
  };
  auto next_b = [&](uint32_t s) {
    const uint32_t step = RING5 ? 2 * OB::BYTES : OB::BYTES, end = smem_lds + RING;
    return s + step >= end ? s + step - (RING5 ? RING : DEPTH * OB::BYTES) : s + step;
  };

  f32x4 acc[F][FN];
#pragma unroll
  for (int i = 0; i < F; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // The B fragment comes first, so that a lane's four results are consecutive
  // columns of one row (l % 16).
  auto product = [&](const u32x4& a, const u32x4& b, f32x4& c) {
    if constexpr (BF) {
      c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b), __builtin_bit_cast(bf16x8, a), c, 0, 0, 0);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(b[e]), __uint_as_float(a[e]), c, 0, 0, 0);
    }
  };

  // A slice is multiplied in four quarters: half hf of its K (0, 0, 1, 1), the
  // upper or lower half of the wave's rows.  A fragments alternate between two
  // buffers by quarter, B fragments by half.  Each quarter reads what the next
  // needs:
  //   quarter 0: A half 0 lower, B half 1 (first part)
  //   quarter 1: A half 1 upper, B half 1 (rest)
  //   quarter 2: A half 1 lower
  //   quarter 3: A half 0 upper and B half 0 of the next slice
  u32x4 a[2][FH], b[2][FN];
  uint32_t va, vb;  // this lane's addresses in the slice being read
  const uint32_t la = OA::lane_base(lane, wm * WT), lb = OB::lane_base(lane, wn * WC);
  auto read = [&](auto q_c, int u) {
    constexpr int q = decltype(q_c)::value;
    if constexpr (q == 3) {  // in the order the next products need them
      if (u == 0) a[0][0] = OA::read(va, 0, 0);
      else if (u <= FN) b[0][u - 1] = OB::read(vb, 0, u - 1);
      else a[0][u - FN] = OA::read(va, 0, u - FN);
    } else if constexpr (q == 0) {
      if (u < FH) a[1][u] = OA::read(va, 0, FH + u);
      else b[1][u - FH] = OB::read(vb, 1, u - FH);
    } else if constexpr (q == 1) {
      if (u < FH) a[0][u] = OA::read(va, 1, u);
      else b[1][FN / 2 + u - FH] = OB::read(vb, 1, FN / 2 + u - FH);
    } else {
      a[1][u] = OA::read(va, 1, FH + u);
    }
  };
  // Quarter q: its products in NSL slots, with its reads and the loads
  // load(0) .. load(ND - 1) spread over them.
  auto quarter = [&](auto q_c, auto nd_c, auto&& load) {
    constexpr int q = decltype(q_c)::value, ND = decltype(nd_c)::value;
    constexpr int NM = FH * FN, NSL = NM < 4 ? NM : 4, MPS = NM / NSL;
    constexpr int NR = q == 3 ? FH + FN : (q == 2 ? FH : FH + FN / 2);
    constexpr int RPS = (NR + NSL - 1) / NSL;
#pragma unroll
    for (int u = 0; u < NSL; ++u) {
#pragma unroll
      for (int d = 0; d < ND; ++d)
        if (u == d * NSL / (ND ? ND : 1)) load(d);
#pragma unroll
      for (int r = u * RPS; r < (u + 1) * RPS && r < NR; ++r) read(q_c, r);
#pragma unroll
      for (int m = u * MPS; m < (u + 1) * MPS; ++m)
        product(a[q & 1][m / FN], b[q >> 1][m % FN], acc[(q & 1) * FH + m / FN][m % FN]);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  using Q0 = std::integral_constant<int, 0>;
  using Q1 = std::integral_constant<int, 1>;
  using Q2 = std::integral_constant<int, 2>;
  using Q3 = std::integral_constant<int, 3>;

  // Pipeline.  Between the third and the fourth quarter of slice t a wave
  // waits for its own loads of slice t + 1 and meets the others: that
  // publishes slice t + 1 and frees slice t's slots (the fourth quarter's
  // fragments are in registers).  Loads, each into slots freed before:
  //   five shared slots:  B of slice t + 1 in the fourth quarter of slice t - 1
  //                       and the first of slice t, A of slice t + 2 in the
  //                       second and third;
  //   DEPTH each:         slice t + DEPTH - 1 in the first three quarters of
  //                       slice t (where slice t - 1 was).
  uint32_t sa = smem_lds, sb = smem_lds + (RING5 ? OA::BYTES : RING_A);   // slots of slice t
  uint32_t wa = sa, wb = sb;                                              // slots loaded next
  constexpr int AHEAD = RING5 ? 2 : DEPTH - 1;                            // slices loaded before the loop
#pragma unroll
  for (int t = 0; t < AHEAD; ++t) {
#pragma unroll
    for (int q = 0; q < DPA; ++q) load_a(t, wa, q);
#pragma unroll
    for (int q = 0; q < (RING5 && t == 1 ? DPB / 2 : DPB); ++q) load_b(t, wb, q);
    if (!RING5) { wa = next_a(wa); wb = next_b(wb); }
    else if (t == 0) { wa = next_a(wa); wb = next_b(wb); }
  }
  wait_vmcnt<RING5 ? DPA + DPB / 2 : (AHEAD - 1) * (DPA + DPB)>();
  __builtin_amdgcn_s_barrier();
  va = la + sa;
  vb = lb + sb;
#pragma unroll
  for (int u = 0; u < FH + FN; ++u) read(Q3{}, u);
  __builtin_amdgcn_sched_barrier(0);
  for (int t = 0; t < KT; ++t) {
    const uint32_t sa1 = next_a(sa), sb1 = next_b(sb);
    if constexpr (RING5) {
      const uint32_t sa2 = next_a(sa1), sb2 = next_b(sb1);
      quarter(Q0{}, std::integral_constant<int, DPB / 2>{}, [&](int d) { load_b(t + 1, sb1, DPB / 2 + d); });
      quarter(Q1{}, std::integral_constant<int, DPA / 2>{}, [&](int d) { load_a(t + 2, sa2, d); });
      quarter(Q2{}, std::integral_constant<int, DPA / 2>{}, [&](int d) { load_a(t + 2, sa2, DPA / 2 + d); });
      wait_vmcnt<DPA>();
      wb = sb2;
    } else {
      quarter(Q0{}, std::integral_constant<int, DPB>{}, [&](int d) { load_b(t + AHEAD, wb, d); });
      quarter(Q1{}, std::integral_constant<int, DPA / 2>{}, [&](int d) { load_a(t + AHEAD, wa, d); });
      quarter(Q2{}, std::integral_constant<int, DPA - DPA / 2>{}, [&](int d) { load_a(t + AHEAD, wa, DPA / 2 + d); });
      wait_vmcnt<(AHEAD - 1) * (DPA + DPB)>();
      wa = next_a(wa);
      wb = next_b(wb);
    }
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): this wave's reads of slice t are done
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    sa = sa1;
    sb = sb1;
    va = la + sa;
    vb = lb + sb;
    if constexpr (RING5)
      quarter(Q3{}, std::integral_constant<int, DPB / 2>{}, [&](int d) { load_b(t + 2, wb, d); });
    else
      quarter(Q3{}, std::integral_constant<int, 0>{}, [&](int) {});
  }
  // Loads past the last slice have landed and every wave is done with the ring.
  wait_vmcnt<0>();
  __syncthreads();

  // Epilogue.  Half the tile's rows at a time (the upper, then the lower half
  // of every wave's) go through LDS as rows of fp32, then a thread finishes 8
  // consecutive columns of a row.
  float* const S = reinterpret_cast<float*>(smem);
  constexpr int HWT = WT / 2;
  constexpr int CPR = BN / 8, RPI = NTH / CPR, NIT = RH / RPI;
  const int c8 = (tid % CPR) * 8, rr0 = tid / CPR;
  const int64_t j = j0 + c8;
  const int valid = j >= p.N ? 0 : (p.N - j < 8 ? (int)(p.N - j) : 8);
  float bias[8];
  if (!p.part) bias8(p, j, valid, bias);
  auto pass = [&](auto pass_c) {
    constexpr int ps = decltype(pass_c)::value;
#pragma unroll
    for (int ii = 0; ii < FH; ++ii)
#pragma unroll
      for (int jj = 0; jj < FN; ++jj)
        *(f32x4*)(S + (wm * HWT + ii * 16 + (lane & 15)) * PITCH + wn * WC + jj * 16 + (lane >> 4) * 4) = acc[ps * FH + ii][jj];
    __syncthreads();
    with_act(p.act, [&](auto act_c) {
      constexpr int ACT = decltype(act_c)::value;
      if (valid > 0) {
#pragma unroll 4
        for (int it = 0; it < NIT; ++it) {
          const int rr = rr0 + it * RPI;
          const int64_t i = i0 + (rr / HWT) * WT + ps * HWT + rr % HWT;
          if (i >= p.M) continue;
          const f32x4 s0 = *(const f32x4*)(S + rr * PITCH + c8), s1 = *(const f32x4*)(S + rr * PITCH + c8 + 4);
          float v[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) { v[e] = s0[e]; v[4 + e] = s1[e]; }
          if (p.part) {
            float* const d = p.part + ((int64_t)sp * p.M + i) * p.ldpart + j;
            *(f32x4*)d = s0;
            *(f32x4*)(d + 4) = s1;
          } else {
            finish8<ACT, BF>(p, i, j, valid, bias, v);
          }
        }
      }
    });
    __syncthreads();
  };
  pass(std::integral_constant<int, 0>{});
  pass(std::integral_constant<int, 1>{});
}

// Split sums: y = epilogue(part[0] + part[1] + ...), chunks in order.
template <bool BF>
__global__ __launch_bounds__(256) void split_finish_kernel(const LinGemm p) {
  const int64_t chunks = p.ldpart / 8;
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t i = at / chunks, j = (at - i * chunks) * 8;
  if (i >= p.M) return;
  const int valid = p.N - j < 8 ? (int)(p.N - j) : 8;
  float v[8], b[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = 0.f;
  const float* src = p.part + i * p.ldpart + j;
#pragma unroll 4
  for (int c = 0; c < p.split; ++c) {
    const f32x4 s0 = *(const f32x4*)src, s1 = *(const f32x4*)(src + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) { v[e] += s0[e]; v[4 + e] += s1[e]; }
    src += p.M * p.ldpart;
  }
  bias8(p, j, valid, b);
  with_act(p.act, [&](auto act_c) { finish8<decltype(act_c)::value, BF>(p, i, j, valid, b, v); });
}

// Copy with zero padding: 64 consecutive lanes take consecutive 16-byte chunks
// of a destination row; a matrix per grid z.
template <typename T>
__global__ __launch_bounds__(256) void pack_kernel(const PackJobs p) {
  constexpr int E = 16 / sizeof(T);
  const PackJob& w = p.job[blockIdx.z];
  const int64_t c = ((int64_t)blockIdx.x * 64 + (threadIdx.x & 63)) * E;
  if (c >= w.ldd) return;
  for (int64_t r = (int64_t)blockIdx.y * 4 + (threadIdx.x >> 6); r < w.rows; r += (int64_t)gridDim.y * 4) {
    const T* s = (const T*)w.src + r * w.lds + c;
    u32x4 o;
    if (c + E <= w.cols) {
      o = load16(s);  // rows may start anywhere
    } else {
      T v[E];
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = c + e < w.cols ? s[e] : T(0);
      __builtin_memcpy(&o, v, 16);
    }
    *(u32x4*)((T*)w.dst + r * w.ldd + c) = o;
  }
}

template <typename T, int KIND, int BM, int BN, int WM, int WN, int DEPTH>
hipError_t launch_tile(const LinGemm& g, hipStream_t s) {
  const int64_t grid = ((g.M + BM - 1) / BM) * ((g.N + BN - 1) / BN) * g.split;
  if (grid <= 0) return hipSuccess;
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  return launch_kernel(linear_tile_kernel<T, KIND, BM, BN, WM, WN, DEPTH>, dim3((unsigned)grid), g, s, WM * WN * 64);
}

template <int KIND>
hipError_t launch_kind(const LinGemm& g, bool bf16, LinTile tile, hipStream_t s) {
  if (bf16) {
    switch (tile) {
      case kTile256: return launch_tile<uint16_t, KIND, 256, 256, 2, 4, 0>(g, s);
      case kTile256x128: return launch_tile<uint16_t, KIND, 256, 128, 4, 2, 3>(g, s);
      case kTile128: return launch_tile<uint16_t, KIND, 128, 128, 2, 2, 0>(g, s);
      default: return launch_tile<uint16_t, KIND, 64, 64, 2, 2, 3>(g, s);
    }
  }
  switch (tile) {
    case kTile256x128: return launch_tile<float, KIND, 256, 128, 4, 2, 3>(g, s);
    case kTile64: return launch_tile<float, KIND, 64, 64, 2, 2, 0>(g, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_linear_tiles(const LinGemm& g, bool bf16, LinKind kind, LinTile tile, hipStream_t s) {
  // What the kernel's loads assume: 16-byte aligned operand rows, and panels
  // and slices within a descriptor's 2^31 bytes.
  const int64_t es = bf16 ? 2 : 4, ch = 16 / es;
  const bool acol = kind == kColCol, bcol = kind != kRowRow;
  if (((uintptr_t)g.A & 15) || ((uintptr_t)g.B & 15) || g.lda % ch || g.ldb % ch) return hipErrorInvalidValue;
  if ((!acol || !bcol) && g.K % ch) return hipErrorInvalidValue;
  if (g.lda * es >= ((int64_t)1 << 23) || g.ldb * es >= ((int64_t)1 << 23)) return hipErrorInvalidValue;
  if (g.split < 1 || (g.split > 1 && !g.part) || (g.part && g.ldpart % 8)) return hipErrorInvalidValue;
  if (kind == kRowRow) return launch_kind<kRowRow>(g, bf16, tile, s);
  if (kind == kRowCol) return launch_kind<kRowCol>(g, bf16, tile, s);
  return launch_kind<kColCol>(g, bf16, tile, s);
}

hipError_t launch_split_finish(const LinGemm& g, bool bf16, hipStream_t s) {
  const int64_t grid = (g.M * (g.ldpart / 8) + 255) / 256;
  if (grid <= 0) return hipSuccess;
  if (grid > INT32_MAX || !g.part) return hipErrorInvalidValue;
  return bf16 ? launch_kernel(split_finish_kernel<true>, dim3((unsigned)grid), g, s)
              : launch_kernel(split_finish_kernel<false>, dim3((unsigned)grid), g, s);
}

hipError_t launch_pack(const PackJobs& p, bool bf16, hipStream_t s) {
  const int64_t e = bf16 ? 8 : 4;
  int64_t gx = 0, gy = 0;
  for (int i = 0; i < p.n; ++i) {
    const PackJob& w = p.job[i];
    if (w.ldd % e || ((uintptr_t)w.dst & 15)) return hipErrorInvalidValue;
    if (!w.rows) continue;
    gx = std::max(gx, (w.ldd / e + 63) / 64);
    gy = std::max(gy, std::min<int64_t>((w.rows + 3) / 4, 65535));
  }
  if (gx <= 0 || gy <= 0) return hipSuccess;
  const dim3 grid((unsigned)gx, (unsigned)gy, (unsigned)p.n);
  return bf16 ? launch_kernel(pack_kernel<uint16_t>, grid, p, s) : launch_kernel(pack_kernel<float>, grid, p, s);
}

}  // namespace muon
