// Product of 8-bit rotated activations with a CQ matrix on the integer matrix
// cores:
//   y[b][n] = s_b * sum over groups g of (norm[n][g] / sqrt(G)) * sum over j in g of q[b][j] * c[n][j]
// with q the activations in the rotated space (orthonormal Hadamard, as the
// 8-bit norm writes them) and c the codebook levels: the orthonormal Hadamard
// matrix is its own inverse, so x_g . W_hat_g is the product of the rotated
// activations with the levels ("Cactus Quants CQ2-bit Quantization: Extreme
// Compression for Edge LLMs", section Hadamard Rotation).
//
// The levels enter as 16-bit whole numbers, c ~ scale * (256 hi + lo), so
// every sum within a group is an exact integer: two v_mfma_i32 per product,
// the hi products' sum shifted up by 8 and added to the lo products' (|sum| <=
// 256 * 128 * 32768 = 2^30 at the largest group).  Only its conversion and the
// step between groups, one fma with the group's norm, round.  Two integer terms
// take the matrix cores as long as one bf16 product of the same shape would,
// and the activations are a quarter of the bytes of float32.
#include <type_traits>

#include "lanes.h"

namespace cq {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void* lds_ptr_t;

__device__ __forceinline__ float half_value(uint32_t h) {
  return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(h)));
}

// Bytes of `bytes` packed codes at any address.
template <int BYTES>
struct Raw {
  uint32_t w[(BYTES + 3) / 4];
};
template <int BYTES>
__device__ __forceinline__ void load_raw(const uint8_t* p, Raw<BYTES>& r) {
  if constexpr (BYTES % 4) r.w[BYTES / 4] = 0;
  __builtin_memcpy(r.w, p, BYTES);
}

// Four codes' selectors, one per byte: selectors() number i of a lane's run,
// in the order in which ordered() puts the activations.
//   3 bits: codes 4i .. 4i + 3.
//   4 bits: of 8 codes the even ones, then the odd ones: two operations
//     spread eight codes instead of ten, at two byte permutes per 8
//     activations.
//   2 bits: codes 4i .. 4i + 3, four operations; or, SHUFFLE, of 16 codes
//     every fourth from code i % 4, seven operations for four selectors, at
//     eight byte permutes per 16 activations.
template <int SB, bool SHUFFLE, int BYTES>
__device__ __forceinline__ uint32_t selectors(const Raw<BYTES>& r, int i) {
  if constexpr (SB == 2 && SHUFFLE) {
    return (r.w[i / 4] >> (2 * (i % 4))) & 0x03030303u;
  } else if constexpr (SB == 2) {
    uint32_t t = __builtin_amdgcn_ubfe(r.w[i / 4], 8 * (i % 4), 8);
    t |= t << 12;
    t |= t << 6;
    return t & 0x03030303u;
  } else if constexpr (SB == 3) {
    const int bit = 12 * i, w = bit / 32, o = bit % 32;
    uint32_t t;
    if (o <= 20)
      t = __builtin_amdgcn_ubfe(r.w[w], o, 12);
    else
      t = __builtin_amdgcn_alignbit(r.w[w + 1 < (BYTES + 3) / 4 ? w + 1 : w], r.w[w], o) & 0xFFFu;
    t = (t | (t << 10)) & 0x003F003Fu;
    return (t | (t << 5)) & 0x07070707u;
  } else {
    return (r.w[i / 2] >> (4 * (i % 2))) & 0x0F0F0F0Fu;
  }
}
// The levels' bytes of four selectors.  At 4 bits the sixteen entries lie in
// two tables of eight: v_perm_b32 takes bytes 0 .. 7 by selectors 0 .. 7 and
// has fixed results for 8 .. 15 (the sign of byte 1, 3, 5, 7 of the table, 0,
// then 255 three times), so
//   entry(i) = permute(first, i) ^ permute(second, i ^ 8)
// once each table holds its entries xor what the other one answers to the
// same code (xor_tables() below).  Three operations instead of five per byte
// lookup and none for a mask.
template <int SB>
__device__ __forceinline__ uint32_t pick(const uint32_t (&t)[4], uint32_t sel) {
  if constexpr (SB == 2) return __builtin_amdgcn_perm(0u, t[0], sel);
  if constexpr (SB == 3) return __builtin_amdgcn_perm(t[1], t[0], sel);
  return __builtin_amdgcn_perm(t[1], t[0], sel) ^ __builtin_amdgcn_perm(t[3], t[2], sel ^ 0x08080808u);
}

__device__ __forceinline__ int byte_perm(int hi, int lo, uint32_t s) {
  return static_cast<int>(__builtin_amdgcn_perm(static_cast<uint32_t>(hi), static_cast<uint32_t>(lo), s));
}
// Activations of 16 columns in the order of selectors().
template <int SB, bool SHUFFLE>
__device__ __forceinline__ i32x4 ordered(i32x4 q) {
  if constexpr (SB == 4) {
    return i32x4{byte_perm(q.y, q.x, 0x06040200u), byte_perm(q.y, q.x, 0x07050301u), byte_perm(q.w, q.z, 0x06040200u),
                 byte_perm(q.w, q.z, 0x07050301u)};
  } else if constexpr (SB == 2 && SHUFFLE) {  // 4 x 4 bytes transposed
    const int a = byte_perm(q.y, q.x, 0x05010400u), b = byte_perm(q.y, q.x, 0x07030602u);
    const int c = byte_perm(q.w, q.z, 0x05010400u), d = byte_perm(q.w, q.z, 0x07030602u);
    return i32x4{byte_perm(c, a, 0x05040100u), byte_perm(c, a, 0x07060302u), byte_perm(d, b, 0x05040100u),
                 byte_perm(d, b, 0x07060302u)};
  } else {
    return q;
  }
}

// ---- Few batch rows -------------------------------------------------------------------

// A block takes 16 outputs and all batch rows (up to 64); its waves take
// consecutive runs of groups and add their sums through LDS in wave order.
//
// v_mfma_i32_16x16x64_i8 multiplies 16 activation rows with 16 outputs over
// 64 columns, a quarter of the columns per 16 lanes.  With up to 8 batch rows
// (P = 2) the 16 activation rows are 2 groups times 8 batch rows: row (p, b)
// holds batch row b in the columns of group p and zeros elsewhere, so a
// product covers two groups (a unit) whose sums stay apart, and they are
// scaled together.  P = 2 with two row tiles serves up to 16 batch rows, P =
// 1 with 2, 3 or 4 up to 64.
//
// The operands' lanes run over rows first, and a load instruction takes a
// cycle per lane where neighbouring lanes meet different lines: with operands
// loaded in place, 4-bit 4096 x 11008 at 37 batch rows spent about 400 cycles
// per group and CU on them (18.7 us in all), 2-bit 11008 x 4096 at 64 rows
// 29.8 us.  So a wave loads a unit's codes and activations in memory order
// (whole lines), one unit ahead, passes them through its own piece of LDS
// (rows an odd number of 16 bytes apart, so that 8 rows of one column fall on
// different banks) and reads the operands there: 14.4 and 18.5 us.  One batch
// row, 2 bits: 4096 x 4096 4.1 us, 11008 x 4096 6.4 (1.9 TB/s of its bytes),
// 32000 x 4096 12.8, or 2.9 us and 0.31 per 1000 outputs.  By the counters the
// vector units are busy for half of the time (3.2 of 6.4 us; 2.4 operations a
// code, the decoding and all else) and the waves wait for loads and LDS for 55%
// of theirs; at 37 rows (4-bit 4096 x 11008, two waves per SIMD) half (7.4 of
// 15 us; 5.6 a code) and 36%.  Each wave takes its units one after the other, so
// what bounds both is the chain of load, store, read and product that so few
// waves do not cover.

// What a wave stages per unit: 16 rows of codes, MT 16 / P rows of
// activations and, for activation rows of the other group, a run of zeros.
template <int SB, int G, int MT, int P>
struct FewStage {
  static constexpr int CL = G * P / 4;              // columns per lane and unit
  static constexpr int CB = CL * SB / 8;            // their code bytes
  static constexpr int kCodeRow = 4 * CB;           // code bytes of an output's unit
  static constexpr int kGroupBytes = G * SB / 8;    // moved in pieces that do not cross groups
  static constexpr int kCodePiece = kGroupBytes % 16 == 0 ? 16 : kGroupBytes % 8 == 0 ? 8 : 4;
  static constexpr int kCodeStride = kCodeRow + (kCodeRow % 32 == 0 ? 16 : kCodeRow < 16 ? 8 : 0);
  static constexpr int kCodeLoads = (16 * kCodeRow / kCodePiece + kWave - 1) / kWave;
  static constexpr int kB = 16 / P;                 // batch rows of a row tile
  static constexpr int kXRow = P * G;
  static constexpr int kXStride = kXRow + 16;
  static constexpr int kXLoads = (MT * kB * kXRow / 16 + kWave - 1) / kWave;
  static constexpr int kZeros = P > 1 ? (CL + 15) / 16 * 16 : 0;
  static constexpr int kXAt = 16 * kCodeStride;
  static constexpr int kZeroAt = kXAt + MT * kB * kXStride;
  static constexpr int kBytes = kZeroAt + kZeros;
};

constexpr int kFewWaves = 8;

template <int BYTES>
struct CodePiece {
  uint32_t w[BYTES / 4];
};

// MT tiles of 16 / P batch rows; W: waves per block.
template <int SB, int G, int MT, int P, int W>
__global__ void __launch_bounds__(W* kWave)
few_kernel(GemmQ8Args a, Q8Levels lv, float unit) {
  using F = FewStage<SB, G, MT, P>;
  constexpr int CL = F::CL, CB = F::CB, kB = F::kB;
  constexpr int S = CL >= 16 ? CL / 16 : 1;   // products per unit and term
  constexpr int SL = CL >= 16 ? 4 : 2;        // dwords per product (2: v_mfma_i32_16x16x32_i8)
  // The activations are reordered once, on their way into LDS; at 2 bits that
  // pays where there are few of them per code.
  constexpr bool SHUFFLE = CL >= 16 && 8 * F::kXLoads < 9 * (CL / 16);
  constexpr int kSums = MT * 4 * kWave;       // a wave's sums, left where its units were
  constexpr int kWaveBytes = F::kBytes > 4 * kSums ? F::kBytes : 4 * kSums;
  static_assert(kWaveBytes % 16 == 0, "every wave's piece starts on 16 bytes");
  __shared__ __attribute__((aligned(16))) uint8_t stage[W * kWaveBytes];
  const int lane = threadIdx.x & (kWave - 1), r = lane & 15, j = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  uint8_t* const mine = stage + wave * kWaveBytes;
  const int p = j * P / 4, piece = j % (4 / P);  // this lane's group of a unit, and its piece of it
  const int ng = static_cast<int>(a.k / G), units = (ng + P - 1) / P;
  const int batch = static_cast<int>(a.batch);
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 16;
  const int per = (units + W - 1) / W;
  const int g0 = wave * per < units ? wave * per : units, g1 = g0 + per < units ? g0 + per : units;
  const int last = a.n_out - n0 < 16 ? static_cast<int>(a.n_out - n0) - 1 : 15;  // last output of the tile
  const int row_bytes = ng * F::kGroupBytes;
  const uint8_t* const tile = a.packed + n0 * row_bytes;
  const uint16_t* const norms = a.norms + (n0 + (r < last ? r : last)) * ng;
  // The scale of this thread's first output, fetched ahead of the sums.
  const int b_first = threadIdx.x / 16 % (MT * kB);
  const float s_first = a.scale[b_first < batch ? b_first : batch - 1];

  // With up to 4 batch rows at P = 2 the later half of the loads holds none of
  // them: not loaded, its activation rows only meet sums that are not stored.
  const bool half = P == 2 && MT == 1 && F::kXLoads % 2 == 0 && batch <= kB / 2;
  // The pieces of a unit this lane moves.
  constexpr int kPer = F::kCodeRow / F::kCodePiece, kPerX = F::kXRow / 16;  // per output, per batch row
  CodePiece<F::kCodePiece> c_reg[F::kCodeLoads];
  i32x4 x_reg[F::kXLoads];
  auto fetch = [&](int g) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < F::kCodeLoads; ++i) {
      const int e = lane + i * kWave, row = e / kPer < last ? e / kPer : last;
      int at = g * F::kCodeRow + e % kPer * F::kCodePiece;
      if (P > 1) at = at < row_bytes ? at : row_bytes - F::kCodePiece;  // the second group may be past the row
      __builtin_memcpy(c_reg[i].w, tile + static_cast<int64_t>(row) * row_bytes + at, F::kCodePiece);
    }
#if defined(__HIP_DEVICE_COMPILE__)
    // Batch rows past the batch are outside the buffer (read as zero).
    // Columns past k are the next row's, or outside; they are scaled by zero.
    const auto src = __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(a.q), 0, static_cast<int>(batch * a.k), 0x00020000);
#pragma unroll
    for (int i = 0; i < F::kXLoads; ++i) {
      if (half && i >= F::kXLoads / 2) break;
      const int e = lane + i * kWave, b = e / kPerX;
      const uint32_t off = b < batch ? static_cast<uint32_t>(b * a.k + e % kPerX * 16 + g * F::kXRow) : 0x80000000u;
      x_reg[i] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(src, off, 0, 0));
    }
#endif
  };
  auto put_loads = [&](auto loads) __attribute__((always_inline)) {
    constexpr int kLoads = decltype(loads)::value;
#pragma unroll
    for (int i = 0; i < F::kCodeLoads; ++i) {
      const int e = lane + i * kWave;
      if (16 * kPer % kWave == 0 || e < 16 * kPer)
        __builtin_memcpy(__builtin_assume_aligned(mine + e / kPer * F::kCodeStride + e % kPer * F::kCodePiece, F::kCodePiece),
                         c_reg[i].w, F::kCodePiece);
    }
    i32x4 x[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int e = lane + i * kWave;
      x[i] = ordered<SB, SHUFFLE>(x_reg[i]);
      if (MT * kB * kPerX % kWave == 0 || e < MT * kB * kPerX)
        *reinterpret_cast<i32x4*>(mine + F::kXAt + e / kPerX * F::kXStride + e % kPerX * 16) = x[i];
    }
    wait_lds_writes();
#pragma unroll
    for (int i = 0; i < F::kCodeLoads; ++i)
#pragma unroll
      for (int d = 0; d < F::kCodePiece / 4; ++d) hold_value(c_reg[i].w[d]);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) hold_values(x[i].x, x[i].y, x[i].z, x[i].w);
  };
  auto put = [&]() __attribute__((always_inline)) {
    if (half)
      put_loads(std::integral_constant<int, (F::kXLoads + 1) / 2>{});
    else
      put_loads(std::integral_constant<int, F::kXLoads>{});
  };
  if constexpr (F::kZeros > 0) {
    const i32x4 zero = {0, 0, 0, 0};
    if (lane < F::kZeros / 16) *reinterpret_cast<i32x4*>(mine + F::kZeroAt + lane * 16) = zero;
    wait_lds_writes();
    hold_values(zero.x, zero.y, zero.z, zero.w);
  }

  float acc[MT][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[m][i] = 0.0f;
  auto product = [](i32x4 av, i32x4 bv, i32x4 c) __attribute__((always_inline)) {
    if constexpr (CL >= 16) {
      return __builtin_amdgcn_mfma_i32_16x16x64_i8(av, bv, c, 0, 0, 0);
    } else {
      typedef int i32x2 __attribute__((ext_vector_type(2)));
      return __builtin_amdgcn_mfma_i32_16x16x32_i8(__builtin_bit_cast(int64_t, (i32x2{av.x, av.y})),
                                                   __builtin_bit_cast(int64_t, (i32x2{bv.x, bv.y})), c, 0, 0, 0);
    }
  };

  // Norms of four groups: lane (j, r) holds output r's of group (first of the
  // quad) + j; one load instruction per four groups.
  uint32_t quad = 0;
  auto fetch_norms = [&](int g) __attribute__((always_inline)) -> uint32_t {
    const int at = g * P + j;
    return norms[at < ng ? at : ng - 1];
  };
  constexpr int kUnitsPerQuad = 4 / P;
  int turn = 0;
  if (g0 < g1) {
    fetch(g0);
    quad = fetch_norms(g0);
  }
  for (int g = g0; g < g1; ++g) {
    put();
    const uint32_t nb = static_cast<uint32_t>(__shfl(static_cast<int>(quad), r + 16 * (turn * P + p), kWave));
    turn = turn + 1 == kUnitsPerQuad ? 0 : turn + 1;
    if (g + 1 < g1) {
      fetch(g + 1);
      if (turn == 0) quad = fetch_norms(g + 1);
    }
    Raw<CB> raw;
    if constexpr (CB % 4) raw.w[CB / 4] = 0;
    __builtin_memcpy(raw.w, __builtin_assume_aligned(mine + r * F::kCodeStride + j * CB, CB % 16 == 0 ? 16 : CB % 8 == 0 ? 8 : CB % 4 == 0 ? 4 : CB % 2 == 0 ? 2 : 1), CB);
    i32x4 ch[MT], cl[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) ch[m] = cl[m] = i32x4{0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < S; ++s) {
      i32x4 hi = {0, 0, 0, 0}, lo = {0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < SL; ++i) {
        const uint32_t sel = selectors<SB, SHUFFLE, CB>(raw, 4 * s + i);
        hi[i] = static_cast<int>(pick<SB>(lv.hi, sel));
        lo[i] = static_cast<int>(pick<SB>(lv.lo, sel));
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const uint8_t* at = mine + F::kXAt + (m * kB + r % kB) * F::kXStride + p * G + piece * CL + 16 * s;
        if (P > 1 && r / kB != p) at = mine + F::kZeroAt + 16 * s;
        i32x4 x;
        if constexpr (CL >= 16) {
          x = *reinterpret_cast<const i32x4*>(at);
        } else {
          const int2 half = *reinterpret_cast<const int2*>(at);
          x = i32x4{half.x, half.y, 0, 0};
        }
        ch[m] = product(x, hi, ch[m]);
        cl[m] = product(x, lo, cl[m]);
      }
    }
    // A weight of zero (a group past the row) adds nothing: the sums are finite.
    const float w = P == 1 || g * P + p < ng ? half_value(nb) : 0.0f;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        acc[m][i] = __builtin_fmaf(w, static_cast<float>((ch[m][i] << 8) + cl[m][i]), acc[m][i]);
    asm volatile("" ::: "memory");  // the next unit is stored after this one's reads
  }
  // Register i of lane (j, r) is activation row 4 j + i, output r.
  float* const sums = reinterpret_cast<float*>(mine);
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) sums[(m * 4 + i) * kWave + lane] = acc[m][i];
  wait_lds_writes();
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) hold_value(acc[m][i]);
  __syncthreads();
  for (int e = threadIdx.x; e < MT * kB * 16; e += W * kWave) {
    const int b = e / 16, c = e % 16;
    const int64_t o = n0 + c;
    if (b >= batch || o >= a.n_out) continue;
    float v = 0.0f;
#pragma unroll
    for (int pp = 0; pp < P; ++pp) {
      const int row = pp * kB + b % kB, at = (b / kB * 4 + row % 4) * kWave + row / 4 * 16 + c;
#pragma unroll
      for (int w = 0; w < W; ++w) v += reinterpret_cast<const float*>(stage + w * kWaveBytes)[at];
    }
    v *= unit * (e == static_cast<int>(threadIdx.x) ? s_first : a.scale[b]);
    if (a.y_bf16)
      store_elem<true>(a.y, b * a.n_out + o, v);
    else
      store_elem<false>(a.y, b * a.n_out + o, v);
  }
}

// ---- Many batch rows ---------------------------------------------------------------------

// Block tile 32 TM batch rows x 128 outputs, 4 waves of 32 outputs each.
// v_mfma_i32_32x32x32_i8: lane l holds batch row l % 32 of the activations
// (from LDS) and output l % 32 of the levels, columns of half l / 32 of the
// group; a wave decodes its outputs' codes once per group for all TM row
// tiles.  The activations' next tile moves by direct-to-LDS loads into the
// other buffer while this one is multiplied; 16-byte chunk c of row r lies at
// slot c ^ chunk_key(r), so that the operand reads, 16 rows of one chunk at a
// time, cover all 64 banks (no conflicts, by the counters).
//
// 4096 rows, 2-bit 11008 x 4096 (3.7e11 operations, twice that in the two
// terms): 361 to 404 us by the clock the card grants, 1.8 to 2.0 POP/s of
// integer operations; a large int8 library product reaches 2.07, the bare
// instruction on random data 3.76.  It took 492 us with the sums scaled before
// the next products instead of beside them, with conflicting chunk slots and
// the blocks in plain order; the bands of output tiles (below) took the L2's
// misses from 1.19e7 to 2.5e6.  What bounds it now are vector operations: a
// wave issues about 320 per step (decoding its outputs' codes, then turning
// each row tile's sums to float32 and scaling them) beside 32 products; they
// keep the vector units busy 65% of the time and the matrix cores 50%.  192
// and 256 rows per block spill registers (432 to 462 us), 256 columns per tile
// took 455.
constexpr int kGemmWaves = 4;
constexpr int kGemmBlock = kGemmWaves * kWave;
constexpr int kGemmCols = 32 * kGemmWaves;
constexpr uint32_t kBand = 8;
__device__ __forceinline__ int chunk_key(int row) { return (row >> 1) & 7; }

template <int SB, int G, int TM>
__global__ void __launch_bounds__(kGemmBlock, 2)
gemm_q8_kernel(GemmQ8Args a, Q8Levels lv, float unit, float* part, int ksplit, int tiles_per) {
  constexpr int BM = 32 * TM;
  constexpr int KT = G > 128 ? G : 128;        // columns per tile
  constexpr int GT = KT / G;                   // groups per tile
  constexpr int S = G / 32;                    // products per group and term
  constexpr int CB = G * SB / 16;              // code bytes per lane and group
  constexpr int CH = KT / 16;                  // 16-byte chunks per row of a tile
  __shared__ __attribute__((aligned(16))) uint8_t xt0[BM * KT];
  __shared__ __attribute__((aligned(16))) uint8_t xt1[BM * KT];
  const int lane = threadIdx.x & (kWave - 1), c32 = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);

  // Consecutive logical blocks run on one XCD.  They go over bands of kBand
  // output tiles, row tile by row tile: the 64 blocks that an XCD runs
  // together share kBand weight tiles and 64 / kBand row tiles, which its L2
  // holds for the whole of k.
  const uint32_t mt = static_cast<uint32_t>((a.batch + BM - 1) / BM);
  const uint32_t lb = xcd_block(blockIdx.x, gridDim.x);
  const uint32_t ks = lb % ksplit, tile = lb / ksplit;
  const uint32_t nt = static_cast<uint32_t>((a.n_out + kGemmCols - 1) / kGemmCols), band = tile / (kBand * mt);
  const uint32_t wide = nt - band * kBand < kBand ? nt - band * kBand : kBand, in_band = tile - band * kBand * mt;
  const uint32_t mtile = in_band / wide, ntile = band * kBand + in_band - mtile * wide;
  const int64_t m0 = static_cast<int64_t>(mtile) * BM;
  const int64_t n = static_cast<int64_t>(ntile) * kGemmCols + 32 * wave + c32;
  const int64_t nc = n < a.n_out ? n : a.n_out - 1;
  const int ng = static_cast<int>(a.k / G);
  const int ntiles = static_cast<int>((a.k + KT - 1) / KT);
  const int t_begin = ks * tiles_per, t_end = t_begin + tiles_per < ntiles ? t_begin + tiles_per : ntiles;
  const uint8_t* const codes = a.packed + nc * ng * (G * SB / 8) + h * CB;
  const uint16_t* const norms = a.norms + nc * ng;

  // Where this lane's pieces of a tile lie, from the tile's first column.
  // Rows past the batch lie outside the buffer (they read zero), columns past
  // k (the last tile at G < 128) are the next row's, or outside: they only
  // meet weights of zero.
  constexpr int kDma = BM * CH / kGemmBlock;
  uint32_t x_off[kDma];
#pragma unroll
  for (int i = 0; i < kDma; ++i) {
    const int slot = (i * kGemmWaves + wave) * kWave + lane, r = slot / CH, c = (slot % CH) ^ chunk_key(r);
    x_off[i] = m0 + r < a.batch ? static_cast<uint32_t>(r * a.k + 16 * c) : 0x80000000u;
  }
  auto issue = [&](int t, uint8_t* dst) __attribute__((always_inline)) {
#if defined(__HIP_DEVICE_COMPILE__)
    const int rows = a.batch - m0 < BM ? static_cast<int>(a.batch - m0) : BM;
    const auto src = __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(a.q + m0 * a.k), 0, rows * static_cast<int>(a.k),
                                                       0x00020000);
#pragma unroll
    for (int i = 0; i < kDma; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (lds_ptr_t)(dst + 16 * ((i * kGemmWaves + wave) * kWave)), 16,
                                               x_off[i] + t * KT, 0, 0, 0);
#endif
  };
  // Groups past k (the last tile at G < 128): the last group's codes, scaled by zero.
  auto load = [&](int t, Raw<CB> (&raw)[GT], uint32_t (&nb)[GT]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < GT; ++i) {
      const int g = t * GT + i, gc = g < ng ? g : ng - 1;
      load_raw<CB>(codes + static_cast<int64_t>(gc) * (G * SB / 8), raw[i]);
      nb[i] = norms[gc];
      if (GT > 1 && g >= ng) nb[i] = 0;
    }
  };

  f32x16 acc[TM];
#pragma unroll
  for (int m = 0; m < TM; ++m) acc[m] = f32x16{};
  Raw<CB> cur[GT], nxt[GT];
  uint32_t ncur[GT], nnxt[GT];

  auto compute = [&](const uint8_t* x) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < GT; ++i) {
      i32x4 hi[S], lo[S];
#pragma unroll
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const uint32_t sel = selectors<SB, false, CB>(cur[i], 4 * s + d);
          hi[s][d] = static_cast<int>(pick<SB>(lv.hi, sel));
          lo[s][d] = static_cast<int>(pick<SB>(lv.lo, sel));
        }
      const float w = half_value(ncur[i]);
      // Row tile m's products are issued before row tile m - 1's sums are
      // scaled, so that the vector operations run beside the matrix cores'.
      i32x16 ch[2], cl[2];
      auto finish = [&](int m) __attribute__((always_inline)) {
#pragma unroll
        for (int e = 0; e < 16; ++e)
          acc[m][e] = __builtin_fmaf(w, static_cast<float>((ch[m & 1][e] << 8) + cl[m & 1][e]), acc[m][e]);
      };
#pragma unroll
      for (int m = 0; m < TM; ++m) {
        const int r = 32 * m + c32;
        ch[m & 1] = cl[m & 1] = i32x16{};
#pragma unroll
        for (int s = 0; s < S; ++s) {
          const int c = i * (G / 16) + h * (G / 32) + s;
          const i32x4 xo = ordered<SB, false>(*reinterpret_cast<const i32x4*>(x + (r * CH + (c ^ chunk_key(r))) * 16));
          ch[m & 1] = __builtin_amdgcn_mfma_i32_32x32x32_i8(xo, hi[s], ch[m & 1], 0, 0, 0);
          cl[m & 1] = __builtin_amdgcn_mfma_i32_32x32x32_i8(xo, lo[s], cl[m & 1], 0, 0, 0);
        }
        if (m > 0) finish(m - 1);
      }
      finish(TM - 1);
    }
  };
  auto step = [&](int t, const uint8_t* x, uint8_t* other) __attribute__((always_inline)) {
    if (t + 1 < t_end) {
      issue(t + 1, other);
      load(t + 1, nxt, nnxt);
    }
    compute(x);
#pragma unroll
    for (int i = 0; i < GT; ++i) {
      cur[i] = nxt[i];
      ncur[i] = nnxt[i];
    }
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): this wave's direct-to-LDS loads
    __syncthreads();
  };

  if (t_begin < t_end) {
    issue(t_begin, xt0);
    load(t_begin, cur, ncur);
  }
  __builtin_amdgcn_s_waitcnt(0x0F70);
  __syncthreads();
  for (int t = t_begin; t < t_end; t += 2) {
    step(t, xt0, xt1);
    if (t + 1 < t_end) step(t + 1, xt1, xt0);
  }

  // Result layout: register e of lane l is batch row 8 (e / 4) + 4 (l / 32) +
  // e % 4 of its row tile, output l % 32.  The rows' scales go through LDS
  // once; every address is a uniform row plus the lane's own offset.
  float* const sc = reinterpret_cast<float*>(xt0);  // all waves are past their last tile
  if (!part) {
    float v = 0.0f;
    if (threadIdx.x < BM) {
      v = m0 + threadIdx.x < a.batch ? unit * a.scale[m0 + threadIdx.x] : 0.0f;
      sc[threadIdx.x] = v;
    }
    wait_lds_writes();
    hold_value(v);
    __syncthreads();
  }
  const bool inside = m0 + BM <= a.batch && static_cast<int64_t>(ntile + 1) * kGemmCols <= a.n_out;  // the whole block tile
  auto uniform_row = [](int m, int e) { return 32 * m + 8 * (e / 4) + e % 4; };
  const uint32_t lane_at = static_cast<uint32_t>(4 * h * a.n_out + n);  // n_out <= 2^27
  float* const to_part = part + (static_cast<int64_t>(ks) * a.batch + m0) * a.n_out;
  uint8_t* const to_y = a.y + m0 * a.n_out * (a.y_bf16 ? 2 : 4);
#pragma unroll
  for (int m = 0; m < TM; ++m) {
    float4 s4[4];
    if (!part) {
#pragma unroll
      for (int i = 0; i < 4; ++i) s4[i] = *reinterpret_cast<const float4*>(sc + 32 * m + 8 * i + 4 * h);
    }
    auto value = [&](int e) __attribute__((always_inline)) {
      const float4& q4 = s4[e / 4];
      return acc[m][e] * (e % 4 == 0 ? q4.x : e % 4 == 1 ? q4.y : e % 4 == 2 ? q4.z : q4.w);
    };
    if (inside && !part && a.y_bf16 && a.n_out % 2 == 0) {
      // Two columns per store: the even lane of a pair stores row e, the odd
      // one row e + 1, each with its neighbour's value.
      const bool odd = lane & 1;
      const uint32_t pair_at = lane_at - odd + (odd ? static_cast<uint32_t>(a.n_out) : 0u);
#pragma unroll
      for (int e = 0; e < 16; e += 2) {
        const float v0 = value(e), v1 = value(e + 1);
        const float mine = odd ? v1 : v0, other = dpp_move<0xB1>(odd ? v0 : v1);
        uint16_t* row = reinterpret_cast<uint16_t*>(to_y) + static_cast<int64_t>(uniform_row(m, e)) * a.n_out;
        *reinterpret_cast<uint32_t*>(row + pair_at) = odd ? pack_bf16(other, mine) : pack_bf16(mine, other);
      }
      continue;
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int row = uniform_row(m, e);
      if (!inside && (n >= a.n_out || m0 + row + 4 * h >= a.batch)) continue;
      if (part)
        (to_part + static_cast<int64_t>(row) * a.n_out)[lane_at] = acc[m][e];
      else if (a.y_bf16)
        (reinterpret_cast<uint16_t*>(to_y) + static_cast<int64_t>(row) * a.n_out)[lane_at] = one_bf16(value(e));
      else
        (reinterpret_cast<float*>(to_y) + static_cast<int64_t>(row) * a.n_out)[lane_at] = value(e);
    }
  }
}

// y from the ksplit partial sums, added in order; zeros from none.
__global__ void __launch_bounds__(256)
gemm_q8_join_kernel(GemmQ8Args a, const float* __restrict__ part, int ksplit, float unit) {
  const int64_t total = a.batch * a.n_out;
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; e < total; e += static_cast<int64_t>(gridDim.x) * 256) {
    float v = 0.0f;
    if (ksplit) {
      v = part[e];
      for (int s = 1; s < ksplit; ++s) v += part[s * total + e];
      v *= unit * a.scale[e / a.n_out];
    }
    if (a.y_bf16)
      store_elem<true>(a.y, e, v);
    else
      store_elem<false>(a.y, e, v);
  }
}

hipError_t launch_join(const GemmQ8Args& a, const float* part, int ksplit, float unit, hipStream_t s) {
  const int64_t blocks = (a.batch * a.n_out + 255) / 256;
  gemm_q8_join_kernel<<<dim3(static_cast<uint32_t>(blocks < most_blocks(256) ? blocks : most_blocks(256))), dim3(256), 0, s>>>(
      a, part, ksplit, unit);
  return hipGetLastError();
}

// Turns 16 bytes (entry i at byte i) into the two tables of pick<4>().
// first[i] = entry[i] ^ answer(second, i ^ 8) and second[i] = entry[8 + i] ^
// answer(first, 8 + i), where answer(t, 8 .. 11) is the sign of t's byte 1,
// 3, 5, 7 as a byte, answer(t, 12) = 0 and answer(t, 13 .. 15) = 255.  Bytes 5
// and 7 depend on no sign, 3 on byte 7's, 1 on byte 3's, the others on these.
void xor_tables(uint32_t (&table)[4]) {
  uint8_t entry[16], t[2][8];
  __builtin_memcpy(entry, table, 16);
  auto answer = [&](int which, int sel) -> uint8_t {
    if (sel >= 13) return 255;
    if (sel == 12) return 0;
    return t[which][2 * (sel - 8) + 1] & 0x80 ? 255 : 0;
  };
  for (const int i : {7, 5, 3, 1, 0, 2, 4, 6})
    for (int which = 0; which < 2; ++which)
      t[which][i] = static_cast<uint8_t>(entry[8 * which + i] ^ answer(1 - which, 8 + i));
  __builtin_memcpy(table, t, 16);
}

// How a call is cut up; the same for the workspace size and the launch.
struct Plan {
  bool few;    // the few-rows kernel
  int ksplit;  // ranges of k
  int per;     // tiles per range
};
// 64 rows: 2-bit 11008 x 4096 18.5 us here and 29.5 tiled, 4-bit 4096 x 11008
// 17.4 and 28.6 (G = 128).  At G = 256 the registers hold 32 rows.
constexpr int64_t kFewRows = 64;
constexpr int kRowTiles = 4;  // row tiles of 32 of the tiled kernel
constexpr int kCus = 256;

int64_t few_blocks(int64_t n_out) { return (n_out + 15) / 16; }
int64_t tile_count(int64_t n_out, int64_t batch) {  // of the tiled kernel, per range of k
  return (n_out + kGemmCols - 1) / kGemmCols * ((batch + 32 * kRowTiles - 1) / (32 * kRowTiles));
}

// The ranges of k that an estimate finds fastest: rounds of one block per CU,
// 1.6 us per tile and block (1.1 to 1.6 measured), two blocks on a CU at 1.7
// times one; then 3 us and 8 bytes per partial sum at 4 TB/s to join them.  Measured (us, ranges
// 1 / 2 / 4 / 8): 2-bit 11008 x 4096 at 128 rows 35.8 / 32.5 / 33.6 / 36.7, at
// 256 37.8 / 46.1 / 47.8 / 67.6; 4-bit 4096 x 11008 at 128 rows 111.7 / 66.7 /
// 42.0 / 30.9, at 256 114.1 / 70.1 / 46.7 / 45.3, at 512 118.8 / 76.6 / 72.4 / 82.6.
Plan plan_for(int64_t n_out, int64_t k, int64_t batch, int group_size) {
  Plan p{};
  p.ksplit = 1;
  if (batch <= (group_size > 128 ? kFewRows / 2 : kFewRows)) {
    p.few = true;
    return p;
  }
  const int kt = group_size > 128 ? group_size : 128;
  const int64_t tiles = (k + kt - 1) / kt;
  const int64_t blocks = tile_count(n_out, batch);
  p.per = static_cast<int>(tiles);
  double best = 0.0;
  // Ranges of 4 tiles or more, and no more than two blocks per CU.
  for (int64_t want = 1; want == 1 || (want <= tiles / 4 && blocks * want <= 2 * kCus); ++want) {
    const int64_t per = (tiles + want - 1) / want, split = (tiles + per - 1) / per;
    const int64_t rounds = (blocks * split + kCus - 1) / kCus;
    const double us = (0.85 * static_cast<double>(rounds / 2 * 2) + static_cast<double>(rounds % 2)) * 1.6 * static_cast<double>(per) +
                      (split > 1 ? 3.0 + static_cast<double>(split) * static_cast<double>(batch * n_out) * 8.0 / 4e6 : 0.0);
    if (want == 1 || us < best) {
      best = us;
      p.per = static_cast<int>(per);
      p.ksplit = static_cast<int>(split);
    }
  }
  return p;
}

template <int SB, int G, int MT, int P>
hipError_t launch_few(const GemmQ8Args& a, const Q8Levels& lv, float unit, hipStream_t s) {
  const dim3 grid(static_cast<uint32_t>(few_blocks(a.n_out)));
  few_kernel<SB, G, MT, P, kFewWaves><<<grid, dim3(kFewWaves * kWave), 0, s>>>(a, lv, unit);
  return hipGetLastError();
}

template <int SB, int G>
hipError_t launch_for(const GemmQ8Args& a, const Q8Levels& lv, const Plan& p, float unit, float* ws, hipStream_t s) {
  if (p.few) {
    if (a.batch <= 8) return launch_few<SB, G, 1, 2>(a, lv, unit, s);
    if (a.batch <= 16) return launch_few<SB, G, 2, 2>(a, lv, unit, s);
    if (a.batch <= 32) return launch_few<SB, G, 2, 1>(a, lv, unit, s);
    if constexpr (G <= 128) {
      if (a.batch <= 48) return launch_few<SB, G, 3, 1>(a, lv, unit, s);
      return launch_few<SB, G, 4, 1>(a, lv, unit, s);
    }
  }
  const int64_t tiles = tile_count(a.n_out, a.batch);
  float* part = p.ksplit > 1 ? ws : nullptr;
  gemm_q8_kernel<SB, G, kRowTiles><<<dim3(static_cast<uint32_t>(tiles * p.ksplit)), dim3(kGemmBlock), 0, s>>>(
      a, lv, unit, part, p.ksplit, p.per);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess && part ? launch_join(a, part, p.ksplit, unit, s) : e;
}

template <int SB>
hipError_t launch_bits(const GemmQ8Args& a, int group_size, const Q8Levels& lv, const Plan& p, float unit, float* ws,
                       hipStream_t s) {
  if (group_size == 32) return launch_for<SB, 32>(a, lv, p, unit, ws, s);
  if (group_size == 64) return launch_for<SB, 64>(a, lv, p, unit, ws, s);
  if (group_size == 128) return launch_for<SB, 128>(a, lv, p, unit, ws, s);
  return launch_for<SB, 256>(a, lv, p, unit, ws, s);
}

}  // namespace

int64_t gemm_q8_workspace(int64_t n_out, int64_t k, int64_t batch, int group_size) {
  if (n_out <= 0 || k <= 0 || batch <= 0) return 0;
  const Plan p = plan_for(n_out, k, batch, group_size);
  return p.ksplit > 1 ? static_cast<int64_t>(p.ksplit) * batch * n_out * 4 : 0;
}

int64_t gemm_q8_threads(int64_t n_out, int64_t k, int64_t batch, int group_size) {
  if (n_out <= 0 || k <= 0 || batch <= 0) return 0;
  const Plan p = plan_for(n_out, k, batch, group_size);
  return p.few ? few_blocks(n_out) * kFewWaves * kWave : tile_count(n_out, batch) * p.ksplit * kGemmBlock;
}

hipError_t launch_gemm_q8_empty(const GemmQ8Args& a, hipStream_t s) {
  return launch_join(a, nullptr, 0, 0.0f, s);
}

hipError_t launch_gemm_q8(const GemmQ8Args& a, int sbits, int group_size, Q8Levels lv, float* ws, hipStream_t s) {
  if (sbits == 4) {
    xor_tables(lv.hi);
    xor_tables(lv.lo);
  }
  const Plan p = plan_for(a.n_out, a.k, a.batch, group_size);
  const float unit = lv.scale / __builtin_sqrtf(static_cast<float>(group_size));
  if (sbits == 2) return launch_bits<2>(a, group_size, lv, p, unit, ws, s);
  if (sbits == 3) return launch_bits<3>(a, group_size, lv, p, unit, ws, s);
  return launch_bits<4>(a, group_size, lv, p, unit, ws, s);
}

}  // namespace cq
