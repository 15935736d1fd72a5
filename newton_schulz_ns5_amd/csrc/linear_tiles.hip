// The linear product and its gradients as tiled MFMA products on gfx950.
//
// C = A B^T with either operand stored K-contiguous ("row") or with its own
// index contiguous ("col"); see LinGemm.  The work is 2 M N K operations on
// operands that are each re-read once per tile of the other, so it is bound by
// the matrix units once a tile is large enough; the kernel is built to keep
// them fed:
//  - one workgroup per BT x BT output tile; BT = 256: eight waves of 128 x 64,
//    two per SIMD; BT = 128 and 64: four waves, two and four workgroups per CU
//    for problems with too few large tiles to fill the chip;
//  - K advances by 128 bytes of a row (64 bf16 or 32 fp32 values) per slice,
//    brought HBM -> LDS directly into a ring of five operand slots, one and a
//    half slices ahead, with one barrier per slice; loads, fragment reads and
//    MFMAs are interleaved in fixed slots;
//  - row operands: a slot row is 128 bytes of K with its 16-byte chunks
//    XOR-swizzled by (row / 2) mod 8, one ds_read_b128 per fragment; col
//    operands: a slot row is one K value of all BT indices, read through the
//    transposing ds_read_b64_tr_b16 (bf16) or single words (fp32).
// Ragged sizes cost nothing in the loop: rows past the end repeat the last one
// (their products are not stored), K values past the end are zeros from the
// buffer descriptor's bounds check (which the loads of the last slice are sent
// past), for both operands, so nothing of a neighbouring buffer enters a sum.
#include "layer_internal.h"
#include "linear_epilogue.h"

namespace muon {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

#define MUON_LDS(p) ((__attribute__((address_space(3))) void*)(p))

constexpr int NSLOT = 5;    // LDS ring of operand slots
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

template <typename T, int KIND, int BT, int NW>
__global__ __launch_bounds__(NW * 64, 1) void linear_tile_kernel(const LinGemm p) {
  constexpr bool BF = sizeof(T) == 2;
  constexpr bool ACOL = KIND == kColCol, BCOL = KIND != kRowRow;
  constexpr int ES = sizeof(T);
  constexpr int KS = ROWB / ES;         // K per slice
  constexpr int NTH = NW * 64;
  constexpr int WT = BT / 2;            // wave tile rows (two rows of waves)
  constexpr int WC = BT / (NW / 2);     // wave tile columns
  constexpr int F = WT / 32, FN = WC / 32;
  constexpr int OPB = BT * ROWB;        // bytes of one slot
  constexpr int DPW = BT / NW / 8;      // load instructions per wave, operand and slice
  constexpr int DQ = DPW / 2;
  constexpr int NM = F * FN;            // block products per quarter slice
  constexpr int MPS = NM >= 8 ? 2 : 1;  // block products per slot
  constexpr int NSL = NM / MPS;
  constexpr int FPS = (F + FN + NSL - 1) / NSL;  // fragment reads per slot
  constexpr int RH = BT / 2;
  constexpr int PITCH = BT + 4;
  constexpr int EPI = RH * PITCH * 4;
  constexpr int LDS_BYTES = NSLOT * OPB > EPI ? NSLOT * OPB : EPI;
  static_assert(DQ >= 1 && DPW % 2 == 0, "a quarter loads half an operand slice");
  __shared__ __attribute__((aligned(16))) uint8_t smem[LDS_BYTES];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / (NW / 2), wn = wave % (NW / 2);
  const int tiles_m = (int)((p.M + BT - 1) / BT), tiles_n = (int)((p.N + BT - 1) / BT);
  int sp, tm, tn;
  decode(tiles_m, tiles_n, sp, tm, tn);
  const int64_t i0 = (int64_t)tm * BT, j0 = (int64_t)tn * BT;

  // This workgroup's slices of K: chunk sp of the split sum.
  const int slices = (int)((p.K + KS - 1) / KS);
  const int t0 = p.split > 1 ? (int)((int64_t)sp * slices / p.split) : 0;
  const int t1 = p.split > 1 ? (int)((int64_t)(sp + 1) * slices / p.split) : slices;
  const int KT = t1 > t0 ? t1 - t0 : 1;             // an empty sum is one slice of zeros
  const int64_t kbeg = (int64_t)t0 * KS;
  const int64_t kend = (int64_t)t1 * KS < p.K ? (int64_t)t1 * KS : p.K;
  const int Kc = (int)(kend - kbeg);                // K values of this workgroup

  // Per operand: base, and each lane's byte offset for each load instruction.
  // Row operand: instruction q of a wave fills slot rows wave * 8 DPW + 8 q ..
  // + 7; lane l lands at row l / 8, chunk l % 8, and fetches the row's chunk
  // (l % 8) ^ ((row / 2) % 8).  Col operand: slot rows are K values, BT ES
  // bytes each.
  constexpr int CROWB = BT * ES, CCH = CROWB / 16, CRPI = 1024 / CROWB;
  static_assert(KS / NW == DPW * CRPI, "a wave's K rows of a col slice take DPW instructions");
  // XOR key of a K row in a col slot, on 32-byte blocks, so that the four rows
  // and two blocks that 32 lanes of a transposing read touch fall on distinct
  // banks (fp32 is read by single words in order and needs none).
  auto ckey = [](int row) { return !BF ? 0 : (BT == 64 ? 2 * ((row >> 1) & 1) : 2 * (row & 3)); };
  int avo[DPW], bvo[DPW];
  const int64_t arows = p.M - i0, brows = p.N - j0;
  const int lda = __builtin_amdgcn_readfirstlane((int)p.lda), ldb = __builtin_amdgcn_readfirstlane((int)p.ldb);
  auto offsets = [&](int (&vo)[DPW], bool col, int ld, int64_t rows) {
#pragma unroll
    for (int q = 0; q < DPW; ++q) {
      if (col) {
        const int row = wave * (KS / NW) + q * CRPI + lane / CCH, c = lane % CCH;
        const int g = ES == 2 ? 2 * ((c >> 1) ^ ckey(row)) + (c & 1) : c;
        vo[q] = row * ld * ES + g * 16;
      } else {
        const int row = wave * 8 * DPW + 8 * q + (lane >> 3);
        const int g = (lane & 7) ^ ((row >> 1) & 7);
        const int src = row < rows ? row : (int)rows - 1;
        vo[q] = src * ld * ES + g * 16;
      }
    }
  };
  offsets(avo, ACOL, lda, arows);
  offsets(bvo, BCOL, ldb, brows);
  // The last slice's loads: row chunks past K go past the descriptor's end.
  const int klast = Kc - (KT - 1) * KS;             // K values of the last slice (0: none)
  auto tail = [&](int vo, int q) {
    const int row = wave * 8 * DPW + 8 * q + (lane >> 3);
    const int g = (lane & 7) ^ ((row >> 1) & 7);
    return g * (16 / ES) < klast ? vo : kOut;
  };
  // A row operand's panel: its descriptor spans the tile's rows from K value
  // kbeg on.  A col operand's: rebased every slice, ending after its last K
  // row's columns (rounded up to whole chunks).
  const char* const Ab = (const char*)p.A + (ACOL ? kbeg * p.lda + i0 : i0 * p.lda + kbeg) * ES;
  const char* const Bb = (const char*)p.B + (BCOL ? kbeg * p.ldb + j0 : j0 * p.ldb + kbeg) * ES;
  auto span = [&](int64_t rows, int64_t ld) {
    const int64_t r = rows < BT ? rows : BT;
    return Kc > 0 ? ((r - 1) * ld + (Kc + 16 / ES - 1) / (16 / ES) * (16 / ES)) * ES : 0;
  };
  const i32x4 ars = rsrc_words(Ab, ACOL ? 0 : span(arows, p.lda));
  const i32x4 brs = rsrc_words(Bb, BCOL ? 0 : span(brows, p.ldb));
  // Scalar arithmetic only (32-bit compares and products), so that the words
  // stay in scalar registers.
  const int kcol = (int)((p.Kcol < kend ? p.Kcol : kend) - kbeg);
  auto col_bytes = [&](int ld, int64_t rows, int left) {
    const int cols = rows < BT ? ((int)rows + 16 / ES - 1) / (16 / ES) * (16 / ES) : BT;
    return left <= 0 ? 0 : (((left < KS ? left : KS) - 1) * ld + cols) * ES;
  };
  const int afull = ACOL ? col_bytes(lda, arows, KS) : 0, alast = ACOL ? col_bytes(lda, arows, kcol - (KT - 1) * KS) : 0;
  const int bfull = BCOL ? col_bytes(ldb, brows, KS) : 0, blast = BCOL ? col_bytes(ldb, brows, kcol - (KT - 1) * KS) : 0;
  auto col_rsrc = [&](const char* base, int ld, int full, int end, int t) {
    const uint64_t a = (uint64_t)base + (uint64_t)(uint32_t)t * (uint32_t)(KS * ld * ES);
    i32x4 r;
    r[0] = (int)(uint32_t)a;
    r[1] = (int)((uint32_t)(a >> 32) & 0xffffu);
    r[2] = t >= KT - 1 ? end : full;
    r[3] = 0x00020000;
    return r;
  };

  const uint32_t smem_lds =
      __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)smem);
  // Load instruction q of operand op (0: A, 1: B) of slice t.  Slices past the
  // last (the pipeline runs ahead) repeat it into slots nobody reads.
  auto dma = [&](int t, int op, int q) {
    const bool last = t >= KT - 1;
    const int tc = last ? KT - 1 : t;
    const uint32_t dst = smem_lds + (uint32_t)(((2 * t + op) % NSLOT) * OPB + (wave * DPW + q) * 1024);
    if (op == 0) {
      if constexpr (ACOL) lds_dma16_asm(col_rsrc(Ab, lda, afull, alast, tc), dst, avo[q], 0);
      else lds_dma16_asm(ars, dst, last ? tail(avo[q], q) : avo[q], tc * ROWB);
    } else {
      if constexpr (BCOL) lds_dma16_asm(col_rsrc(Bb, ldb, bfull, blast, tc), dst, bvo[q], 0);
      else lds_dma16_asm(brs, dst, last ? tail(bvo[q], q) : bvo[q], tc * ROWB);
    }
  };
  auto slot = [&](int t, int op) { return smem + ((2 * t + op) % NSLOT) * OPB; };

  // A fragment: 16 bytes of K per lane for index l % 32 of a 32-block: bf16,
  // the K values 16 ks + 8 (l / 32) .. + 7 of one 32x32x16 product; fp32, the K
  // values 4 (2 ks + l / 32) .. + 3, one for each of four 32x32x2 products.
  const int h = lane >> 5, r32 = lane & 31;
  const int trow = (8 * h + ((lane & 15) >> 2)) * CROWB;
  auto frag = [&](bool col, int t, int op, int ks, int at) -> u32x4 {
    if (!col) {
      const int so = ((2 * ks + h) ^ ((r32 >> 1) & 7)) * 16;
      return *(const u32x4*)(slot(t, op) + (at + r32) * ROWB + so);
    }
    if constexpr (BF) {
      // Lane l of 16-lane group supplies row 8 h + (l % 16) / 4 (+ 4) of the 16
      // K rows and four columns; the transposing read hands it column l % 32.
      const int row = (lane & 15) >> 2;
      const int blk = ((at >> 4) + ((lane >> 4) & 1)) ^ ckey(row);
      const uint8_t* base = slot(t, op) + 16 * ks * CROWB + trow + blk * 32 + (lane & 3) * 8;
      typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)MUON_LDS(base));
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)MUON_LDS(base + 4 * CROWB));
      return __builtin_bit_cast(u32x4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      const uint8_t* base = slot(t, op) + 4 * (2 * ks + h) * CROWB + (at + r32) * 4;
      u32x4 v;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = *(const uint32_t*)(base + e * CROWB);
      return v;
    }
  };
  // Fragment u (0 .. F + FN - 1) of quarter ks, in the order the products need
  // them: a[0], b[0 .. FN - 1], a[1 .. F - 1].
  auto read = [&](int t, int ks, int u, u32x4 (&a)[F], u32x4 (&b)[FN]) {
    if (u == 0) a[0] = frag(ACOL, t, 0, ks, wm * WT);
    else if (u <= FN) b[u - 1] = frag(BCOL, t, 1, ks, wn * WC + (u - 1) * 32);
    else a[u - FN] = frag(ACOL, t, 0, ks, wm * WT + (u - FN) * 32);
  };

  f32x16 acc[F][FN];
#pragma unroll
  for (int i = 0; i < F; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;

  auto product = [&](const u32x4& a, const u32x4& b, f32x16& c) {
    if constexpr (BF) {
      c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a[e]), __uint_as_float(b[e]), c, 0, 0, 0);
    }
  };
  // One quarter of a slice: its products on (ac, bc); the first slots also read
  // the next quarter's fragments (of slice rt) into (an, bn), and load
  // instructions q0 .. q0 + DQ - 1 of operand dop of slice dt are spread over
  // the slots.
  auto quarter = [&](int rt, int rks, u32x4 (&an)[F], u32x4 (&bn)[FN], const u32x4 (&ac)[F], const u32x4 (&bc)[FN],
                     int dt, int dop, int q0) {
#pragma unroll
    for (int u = 0; u < NSL; ++u) {
#pragma unroll
      for (int q = 0; q < DQ; ++q)
        if (u == (q * NSL) / DQ) dma(dt, dop, q0 + q);
#pragma unroll
      for (int f = u * FPS; f < (u + 1) * FPS && f < F + FN; ++f) read(rt, rks, f, an, bn);
#pragma unroll
      for (int m = u * MPS; m < (u + 1) * MPS; ++m) product(ac[m / FN], bc[m % FN], acc[m / FN][m % FN]);
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // Pipeline.  Step t multiplies slice t in four quarters; between the third
  // and the fourth it waits for its own loads of slice t + 1 and meets the
  // other waves, which publishes slice t + 1 and frees slice t's slots.
  //   last quarter of step t - 1, first of step t:  B of slice t + 1
  //   second and third quarter of step t:           A of slice t + 2
  u32x4 a0[F], b0[FN], a1[F], b1[FN];
#pragma unroll
  for (int q = 0; q < DPW; ++q) dma(0, 0, q);
#pragma unroll
  for (int q = 0; q < DPW; ++q) dma(0, 1, q);
#pragma unroll
  for (int q = 0; q < DPW; ++q) dma(1, 0, q);
#pragma unroll
  for (int q = 0; q < DQ; ++q) dma(1, 1, q);
  wait_vmcnt<DPW + DQ>();
  __builtin_amdgcn_s_barrier();
#pragma unroll
  for (int u = 0; u < F + FN; ++u) read(0, 0, u, a0, b0);
  __builtin_amdgcn_sched_barrier(0);
  for (int t = 0; t < KT; ++t) {
    quarter(t, 1, a1, b1, a0, b0, t + 1, 1, DQ);
    quarter(t, 2, a0, b0, a1, b1, t + 2, 0, 0);
    quarter(t, 3, a1, b1, a0, b0, t + 2, 0, DQ);
    wait_vmcnt<DPW>();
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): this wave's reads of slice t are done
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    quarter(t + 1, 0, a0, b0, a1, b1, t + 2, 1, 0);
  }
  // Loads past the last slice have landed and every wave is done with the ring.
  wait_vmcnt<0>();
  __syncthreads();

  // Epilogue.  Register e of a 32 x 32 block holds row 8 (e / 4) + 4 h + e % 4,
  // column l % 32.  Half the tile's rows at a time (the upper, then the lower
  // half of every wave's) go through LDS as rows of fp32, then a thread
  // finishes 8 consecutive columns of a row.
  float* const S = reinterpret_cast<float*>(smem);
  constexpr int HWT = WT / 2;
  constexpr int CPR = BT / 8, RPI = NTH / CPR, NIT = RH / RPI;
  const int c8 = (tid % CPR) * 8, rr0 = tid / CPR;
  const int64_t j = j0 + c8;
  const int valid = j >= p.N ? 0 : (p.N - j < 8 ? (int)(p.N - j) : 8);
  float bias[8];
  if (!p.part) bias8(p, j, valid, bias);
  auto pass = [&](auto pass_c) {
    constexpr int ps = decltype(pass_c)::value;
    // F == 1: a wave's 32 rows are split between the passes by register.
#pragma unroll
    for (int ii = 0; ii < (F + 1) / 2; ++ii)
#pragma unroll
      for (int jj = 0; jj < FN; ++jj)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          if (F == 1 && (e >> 3) != ps) continue;
          const int blk = F == 1 ? 0 : ps * (F / 2) + ii;
          const int row = 8 * (e >> 2) + 4 * h + (e & 3) - (F == 1 ? 16 * ps : 0);
          S[(wm * HWT + ii * 32 + row) * PITCH + wn * WC + jj * 32 + r32] = acc[blk][jj][e];
        }
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

// Copy with zero padding: consecutive lanes take consecutive 16-byte chunks of
// the destination.
template <typename T>
__global__ __launch_bounds__(256) void pack_kernel(const PackJobs p) {
  constexpr int E = 16 / sizeof(T);
  int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (at >= p.start[p.n]) return;
  const int q = p.n > 1 && at >= p.start[1];
  const PackJob& w = p.job[q];
  at -= p.start[q];
  const int64_t per = w.ldd / E, r = at / per, c = (at - r * per) * E;
  const T* s = (const T*)w.src + r * w.lds + c;
  T v[E];
#pragma unroll
  for (int e = 0; e < E; ++e) v[e] = c + e < w.cols ? s[e] : T(0);
  u32x4 o;
  __builtin_memcpy(&o, v, 16);
  *(u32x4*)((T*)w.dst + r * w.ldd + c) = o;
}

template <typename T, int KIND, int BT, int NW>
hipError_t launch_tile(const LinGemm& g, hipStream_t s) {
  const int64_t grid = ((g.M + BT - 1) / BT) * ((g.N + BT - 1) / BT) * g.split;
  if (grid <= 0) return hipSuccess;
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  return launch_kernel(linear_tile_kernel<T, KIND, BT, NW>, dim3((unsigned)grid), g, s, NW * 64);
}

template <int KIND>
hipError_t launch_kind(const LinGemm& g, bool bf16, int tile, hipStream_t s) {
  if (bf16) {
    if (tile == 256) return launch_tile<uint16_t, KIND, 256, 8>(g, s);
    if (tile == 128) return launch_tile<uint16_t, KIND, 128, 4>(g, s);
    return launch_tile<uint16_t, KIND, 64, 4>(g, s);
  }
  if (tile == 128) return launch_tile<float, KIND, 128, 4>(g, s);
  return launch_tile<float, KIND, 64, 4>(g, s);
}

}  // namespace

hipError_t launch_linear_tiles(const LinGemm& g, bool bf16, LinKind kind, int tile, hipStream_t s) {
  // What the kernel's loads assume: 16-byte aligned operand rows, and panels
  // and slices within a descriptor's 2^31 bytes.
  const int64_t es = bf16 ? 2 : 4, ch = 16 / es;
  const bool acol = kind == kColCol, bcol = kind != kRowRow;
  if (((uintptr_t)g.A & 15) || ((uintptr_t)g.B & 15) || g.lda % ch || g.ldb % ch) return hipErrorInvalidValue;
  if ((!acol || !bcol) && g.K % ch) return hipErrorInvalidValue;
  if (g.lda * es >= ((int64_t)1 << 23) || g.ldb * es >= ((int64_t)1 << 23)) return hipErrorInvalidValue;
  if (g.split < 1 || (g.split > 1 && !g.part) || (g.part && g.ldpart % 8)) return hipErrorInvalidValue;
  if (tile != 256 && tile != 128 && tile != 64) return hipErrorInvalidValue;
  if (!bf16 && tile == 256) return hipErrorInvalidValue;
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

hipError_t launch_pack(PackJobs& p, bool bf16, hipStream_t s) {
  const int64_t e = bf16 ? 8 : 4;
  p.start[0] = 0;
  for (int i = 0; i < p.n; ++i) {
    if (p.job[i].ldd % e || ((uintptr_t)p.job[i].dst & 15)) return hipErrorInvalidValue;
    p.start[i + 1] = p.start[i] + p.job[i].rows * (p.job[i].ldd / e);
  }
  const int64_t grid = (p.start[p.n] + 255) / 256;
  if (grid <= 0) return hipSuccess;
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  return bf16 ? launch_kernel(pack_kernel<uint16_t>, dim3((unsigned)grid), p, s)
              : launch_kernel(pack_kernel<float>, dim3((unsigned)grid), p, s);
}

}  // namespace muon
