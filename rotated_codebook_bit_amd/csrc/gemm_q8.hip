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
// the hi products' sum shifted up by 8 as the lo products' starting value
// (|sum| <= 256 * 128 * 32768 = 2^30 at the largest group).  Only the step
// between groups, one fma with the group's norm, rounds.  The two terms cost
// two thirds of what split-bf16 activations and levels cost on the same
// cores at half their rate each, and the activations are a quarter of the
// bytes of float32.
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

// Four codes' selectors (one per byte) and the levels' bytes they select.
// Codes 4i .. 4i + 3 of a lane's run, in the order in which ordered() puts
// the activations: the natural one for 2 and 3 bits; at 4 bits the even
// codes of 8, then the odd ones (two operations instead of five to spread
// eight codes).
template <int SB, int BYTES>
__device__ __forceinline__ uint32_t selectors(const Raw<BYTES>& r, int i) {
  if constexpr (SB == 2) {
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
template <int SB>
__device__ __forceinline__ uint32_t pick(const uint32_t (&t)[4], uint32_t sel) {
  if constexpr (SB == 2) return __builtin_amdgcn_perm(0u, t[0], sel);
  if constexpr (SB == 3) return __builtin_amdgcn_perm(t[1], t[0], sel);
  // Sixteen entries: both halves by the low three bits, then one by the top bit.
  const uint32_t s7 = sel & 0x07070707u, m8 = sel & 0x08080808u, mask = (m8 << 5) - (m8 >> 3);
  const uint32_t a = __builtin_amdgcn_perm(t[1], t[0], s7), b = __builtin_amdgcn_perm(t[3], t[2], s7);
  return (b & mask) | (a & ~mask);
}

// Activations of 16 columns in the order of selectors().
template <int SB>
__device__ __forceinline__ i32x4 ordered(i32x4 q) {
  if constexpr (SB == 4) {
    auto perm = [](int hi, int lo, uint32_t s) {
      return static_cast<int>(__builtin_amdgcn_perm(static_cast<uint32_t>(hi), static_cast<uint32_t>(lo), s));
    };
    return i32x4{perm(q.y, q.x, 0x06040200u), perm(q.y, q.x, 0x07050301u), perm(q.w, q.z, 0x06040200u),
                 perm(q.w, q.z, 0x07050301u)};
  } else {
    return q;
  }
}

// ---- Few batch rows -------------------------------------------------------------------

// A block takes 16 outputs and up to 16 MT batch rows; its 8 waves take
// consecutive runs of groups and add their sums through LDS in wave order.
// v_mfma_i32_16x16x64_i8: lane l holds batch row l % 16 and output l % 16,
// columns of quarter l / 16 of the group, so each lane's codes of a group are
// one load of G SB / 32 bytes (at G = 32 v_mfma_i32_16x16x32_i8).
constexpr int kFewWaves = 8;
constexpr int kFewBlock = kFewWaves * kWave;

template <int SB, int G, int MT, int U>
__global__ void __launch_bounds__(kFewBlock)
few_kernel(GemmQ8Args a, Q8Levels lv, float unit) {
  constexpr int CB = G * SB / 32;             // code bytes per lane and group
  constexpr int S = G >= 64 ? G / 64 : 1;     // products per group and term
  constexpr int CL = G / 4;                   // columns per lane and group
  __shared__ float part[kFewWaves][MT * 256];
  const int lane = threadIdx.x & (kWave - 1), r = lane & 15, j = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int ng = static_cast<int>(a.k / G);
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 16, b0 = static_cast<int64_t>(blockIdx.y) * (16 * MT);
  const int64_t n = n0 + r < a.n_out ? n0 + r : a.n_out - 1;
  const uint8_t* const codes = a.packed + n * ng * (G * SB / 8) + j * CB;
  const uint16_t* const norms = a.norms + n * ng;
  const int8_t* q[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int64_t b = b0 + 16 * m + r;
    q[m] = a.q + (b < a.batch ? b : a.batch - 1) * a.k + j * CL;
  }
  const int per = (ng + kFewWaves - 1) / kFewWaves;
  const int g0 = wave * per < ng ? wave * per : ng, g1 = g0 + per < ng ? g0 + per : ng;

  float acc[MT][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[m][i] = 0.0f;

  for (int g = g0; g < g1; g += U) {
    Raw<CB> raw[U];
    uint32_t nb[U];
    i32x4 x[U][MT][S];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int gu = g + u < g1 ? g + u : g1 - 1;  // past the run: loaded again, scaled by zero
      load_raw<CB>(codes + static_cast<int64_t>(gu) * (G * SB / 8), raw[u]);
      nb[u] = norms[gu];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int s = 0; s < S; ++s) {
          const int8_t* p = q[m] + static_cast<int64_t>(gu) * G + 16 * s;
          if constexpr (G >= 64) {
            x[u][m][s] = *reinterpret_cast<const i32x4*>(p);
          } else {
            const int2 h = *reinterpret_cast<const int2*>(p);
            x[u][m][s] = i32x4{h.x, h.y, 0, 0};
          }
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      i32x4 hi[S], lo[S];
#pragma unroll
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int i = 0; i < (G >= 64 ? 4 : 2); ++i) {
          const uint32_t sel = selectors<SB, CB>(raw[u], 4 * s + i);
          hi[s][i] = static_cast<int>(pick<SB>(lv.hi, sel));
          lo[s][i] = static_cast<int>(pick<SB>(lv.lo, sel));
        }
      const float w = g + u < g1 ? half_value(nb[u]) : 0.0f;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        i32x4 t = {0, 0, 0, 0};
        auto product = [](i32x4 av, i32x4 bv, i32x4 c) __attribute__((always_inline)) {
          if constexpr (G >= 64) {
            return __builtin_amdgcn_mfma_i32_16x16x64_i8(av, bv, c, 0, 0, 0);
          } else {
            typedef int i32x2 __attribute__((ext_vector_type(2)));
            return __builtin_amdgcn_mfma_i32_16x16x32_i8(__builtin_bit_cast(int64_t, (i32x2{av.x, av.y})),
                                                         __builtin_bit_cast(int64_t, (i32x2{bv.x, bv.y})), c, 0, 0, 0);
          }
        };
        i32x4 xo[S];
#pragma unroll
        for (int s = 0; s < S; ++s) {
          xo[s] = ordered<SB>(x[u][m][s]);
          t = product(xo[s], hi[s], t);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) t[i] <<= 8;
#pragma unroll
        for (int s = 0; s < S; ++s) t = product(xo[s], lo[s], t);
        // A norm of zero (a run's end, a zero group) adds nothing, whatever
        // the sum; integers are finite.
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][i] = __builtin_fmaf(w, static_cast<float>(t[i]), acc[m][i]);
      }
    }
  }
  // Result layout: register i of lane l is batch row 4 (l / 16) + i, output l % 16.
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) part[wave][m * 256 + (4 * j + i) * 16 + r] = acc[m][i];
  wait_lds_writes();
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) hold_value(acc[m][i]);
  __syncthreads();
  for (int e = threadIdx.x; e < MT * 256; e += kFewBlock) {
    float v = part[0][e];
#pragma unroll
    for (int w = 1; w < kFewWaves; ++w) v += part[w][e];
    const int64_t b = b0 + e / 16, o = n0 + e % 16;
    if (b >= a.batch || o >= a.n_out) continue;
    v *= unit * a.scale[b];
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
// slot c ^ (r & 7), so the operand reads (8 rows of one chunk) cover all
// banks.
constexpr int kGemmWaves = 4;
constexpr int kGemmBlock = kGemmWaves * kWave;
constexpr int kGemmCols = 32 * kGemmWaves;

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

  // Consecutive logical blocks run on one XCD and share a weight tile.
  const uint32_t mt = static_cast<uint32_t>((a.batch + BM - 1) / BM);
  const uint32_t lb = xcd_block(blockIdx.x, gridDim.x);
  const uint32_t ks = lb % ksplit, tile = lb / ksplit;
  const uint32_t ntile = tile / mt, mtile = tile - ntile * mt;
  const int64_t m0 = static_cast<int64_t>(mtile) * BM;
  const int64_t n = static_cast<int64_t>(ntile) * kGemmCols + 32 * wave + c32;
  const int64_t nc = n < a.n_out ? n : a.n_out - 1;
  const int ng = static_cast<int>(a.k / G);
  const int ntiles = static_cast<int>((a.k + KT - 1) / KT);
  const int t_begin = ks * tiles_per, t_end = t_begin + tiles_per < ntiles ? t_begin + tiles_per : ntiles;
  const uint8_t* const codes = a.packed + nc * ng * (G * SB / 8) + h * CB;
  const uint16_t* const norms = a.norms + nc * ng;

  auto issue = [&](int t, uint8_t* dst) __attribute__((always_inline)) {
#if defined(__HIP_DEVICE_COMPILE__)
    const int rows = a.batch - m0 < BM ? static_cast<int>(a.batch - m0) : BM;
    const int k = static_cast<int>(a.k);
    const auto src = __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(a.q + m0 * a.k), 0, rows * k, 0x00020000);
#pragma unroll
    for (int i = 0; i < BM * CH / kGemmBlock; ++i) {
      const int slot0 = (i * kGemmWaves + wave) * kWave, slot = slot0 + lane;
      const int r = slot / CH, c = (slot % CH) ^ (r & 7);
      // Rows past the batch and columns past k are fetched from outside the
      // buffer: they read zero.
      const int col = t * KT + 16 * c;
      const uint32_t off = r < rows && col < k ? static_cast<uint32_t>(r * k + col) : 0x80000000u;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (lds_ptr_t)(dst + 16 * slot0), 16, off, 0, 0, 0);
    }
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
          const uint32_t sel = selectors<SB, CB>(cur[i], 4 * s + d);
          hi[s][d] = static_cast<int>(pick<SB>(lv.hi, sel));
          lo[s][d] = static_cast<int>(pick<SB>(lv.lo, sel));
        }
      const float w = half_value(ncur[i]);
#pragma unroll
      for (int m = 0; m < TM; ++m) {
        const int r = 32 * m + c32;
        i32x4 xo[S];
#pragma unroll
        for (int s = 0; s < S; ++s) {
          const int c = i * (G / 16) + h * (G / 32) + s;
          xo[s] = ordered<SB>(*reinterpret_cast<const i32x4*>(x + (r * CH + (c ^ (r & 7))) * 16));
        }
        i32x16 t = {};
#pragma unroll
        for (int s = 0; s < S; ++s) t = __builtin_amdgcn_mfma_i32_32x32x32_i8(xo[s], hi[s], t, 0, 0, 0);
#pragma unroll
        for (int e = 0; e < 16; ++e) t[e] <<= 8;
#pragma unroll
        for (int s = 0; s < S; ++s) t = __builtin_amdgcn_mfma_i32_32x32x32_i8(xo[s], lo[s], t, 0, 0, 0);
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[m][e] = __builtin_fmaf(w, static_cast<float>(t[e]), acc[m][e]);
      }
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

  // Result layout: register e of lane l is batch row 8 (e / 4) + 4 (l / 32) + e % 4, output l % 32.
  if (n >= a.n_out) return;
#pragma unroll
  for (int m = 0; m < TM; ++m)
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int64_t b = m0 + 32 * m + 8 * (e / 4) + 4 * h + e % 4;
      if (b >= a.batch) continue;
      if (part) {
        part[(static_cast<int64_t>(ks) * a.batch + b) * a.n_out + n] = acc[m][e];
        continue;
      }
      const float v = acc[m][e] * (unit * a.scale[b]);
      if (a.y_bf16)
        store_elem<true>(a.y, b * a.n_out + n, v);
      else
        store_elem<false>(a.y, b * a.n_out + n, v);
    }
}

// y from the ksplit partial sums, added in order; zeros from none.
__global__ void __launch_bounds__(256)
gemm_q8_join_kernel(GemmQ8Args a, const float* __restrict__ part, int ksplit, float unit) {
  const int64_t total = a.batch * a.n_out;
  const int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (e >= total) return;
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

hipError_t launch_join(const GemmQ8Args& a, const float* part, int ksplit, float unit, hipStream_t s) {
  gemm_q8_join_kernel<<<dim3(static_cast<uint32_t>((a.batch * a.n_out + 255) / 256)), dim3(256), 0, s>>>(a, part, ksplit,
                                                                                                         unit);
  return hipGetLastError();
}

// How a call is cut up; the same for the workspace size and the launch.
struct Plan {
  int few;     // row tiles of 16 of the few-rows kernel, 0: the tiled kernel
  int tm;      // row tiles of 32
  int ksplit;  // ranges of k
  int per;     // tiles per range
};
constexpr int64_t kFewRows = 64;
constexpr int kCus = 256;

Plan plan_for(int64_t n_out, int64_t k, int64_t batch, int group_size) {
  Plan p{};
  p.ksplit = 1;
  if (batch <= kFewRows) {
    p.few = static_cast<int>((batch + 15) / 16);
    return p;
  }
  p.tm = batch <= 64 ? 2 : 4;
  const int kt = group_size > 128 ? group_size : 128;
  const int64_t tiles = (k + kt - 1) / kt;
  const int64_t blocks = (n_out + kGemmCols - 1) / kGemmCols * ((batch + 32 * p.tm - 1) / (32 * p.tm));
  // Fewer blocks than two per CU: ranges of k, at least 8 tiles each.
  int64_t split = blocks < 2 * kCus ? 2 * kCus / blocks : 1;
  if (split > tiles / 8) split = tiles / 8;
  if (split < 1) split = 1;
  p.per = static_cast<int>((tiles + split - 1) / split);
  p.ksplit = static_cast<int>((tiles + p.per - 1) / p.per);
  return p;
}

template <int SB, int G>
hipError_t launch_for(const GemmQ8Args& a, const Q8Levels& lv, const Plan& p, float unit, float* ws, hipStream_t s) {
  if (p.few) {
    const dim3 grid(static_cast<uint32_t>((a.n_out + 15) / 16), 1), block(kFewBlock);
    constexpr int U = G >= 128 ? 2 : 4;
    if (p.few == 1)
      few_kernel<SB, G, 1, 2 * U><<<grid, block, 0, s>>>(a, lv, unit);
    else if (p.few == 2)
      few_kernel<SB, G, 2, U><<<grid, block, 0, s>>>(a, lv, unit);
    else if (p.few == 3)
      few_kernel<SB, G, 3, U><<<grid, block, 0, s>>>(a, lv, unit);
    else
      few_kernel<SB, G, 4, U><<<grid, block, 0, s>>>(a, lv, unit);
    return hipGetLastError();
  }
  const int64_t tiles = (a.n_out + kGemmCols - 1) / kGemmCols * ((a.batch + 32 * p.tm - 1) / (32 * p.tm));
  float* part = p.ksplit > 1 ? ws : nullptr;
  gemm_q8_kernel<SB, G, 4><<<dim3(static_cast<uint32_t>(tiles * p.ksplit)), dim3(kGemmBlock), 0, s>>>(
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

hipError_t launch_gemm_q8_empty(const GemmQ8Args& a, hipStream_t s) {
  return launch_join(a, nullptr, 0, 0.0f, s);
}

hipError_t launch_gemm_q8(const GemmQ8Args& a, int sbits, int group_size, const Q8Levels& lv, float* ws,
                          hipStream_t s) {
  const Plan p = plan_for(a.n_out, a.k, a.batch, group_size);
  const float unit = lv.scale / __builtin_sqrtf(static_cast<float>(group_size));
  if (sbits == 2) return launch_bits<2>(a, group_size, lv, p, unit, ws, s);
  if (sbits == 3) return launch_bits<3>(a, group_size, lv, p, unit, ws, s);
  return launch_bits<4>(a, group_size, lv, p, unit, ws, s);
}

}  // namespace cq
