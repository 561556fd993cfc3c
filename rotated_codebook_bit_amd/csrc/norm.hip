// Residual addition with the root-mean-square norm, in floating point or
// rotated and held in 8 bits for the CQ products, and its gradient.
//
// Forward, per row of n values: h = x + r, y = h * rsqrt(mean(h^2) + eps) * w.
// All of it is float32, from one read of x and r: the row stays in the
// registers of the lanes that loaded it (a wave, 4 or 16 waves per row by its
// width), so h is normalised before it is rounded to its stored type.
//
// 8-bit form: every G-group of y is rotated by the orthonormal Hadamard
// matrix, as the products rotate their activations ("Cactus Quants CQ2-bit
// Quantization: Extreme Compression for Edge LLMs", section Hadamard
// Rotation), the row's largest magnitude m gives the scale s = m / 127, and
// q = round(rotated / s).  One scale per row rather than per group: it leaves
// the products one multiplication per output, and the rotation has already
// spread each group's outliers.
//
// Gradient, with u = w * dy, r = rsqrt(mean(h^2) + eps):
//   dx = dsum + r (u - h r (r mean(u h))),   dw = sum over rows of dy h r.
// In these factors: h r and r mean(u h) are about 1 and u whatever the row's
// magnitude, while r^3 would leave float32 for rows below 1e-13 or above 1e15.
//
// Memory bounds all three at many rows, so nothing is read or written twice
// and every load and store is 16 bytes per lane.  bf16 8192 x 4096 to 8 bits
// with the sum (235 MB) 42.3 us, 5.6 TB/s, where a large copy reaches 4.8;
// float32 16384 x 512 (134 MB) 20.5 us; the gradient of bf16 8192 x 4096 (268
// MB) 49.5 us and 4.8 to add the 512 blocks' shares of dw, 4.9 TB/s.  Few rows
// cost latency: one row of 4096 to 8 bits 3.3 us (a load, two block
// reductions, a store), the gradient of float32 300 x 1000 3.6 us and 3.9.
#include <type_traits>

#include "lanes.h"

namespace cq {
namespace {

// Sum (and max) over the waves of a block: each wave's value through LDS, added
// in wave order by every thread, so the result is the same everywhere.
template <int WAVES>
__device__ __forceinline__ float block_sum(float v, float* red) {
  v = wave_sum(v);
  if constexpr (WAVES > 1) {
    if ((threadIdx.x & (kWave - 1)) == 0) red[threadIdx.x / kWave] = v;
    wait_lds_writes();
    hold_value(v);
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int i = 1; i < WAVES; ++i) v += red[i];
  }
  return v;
}
template <int WAVES>
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* red) {
  v = wave_max(v);
  if constexpr (WAVES > 1) {
    if ((threadIdx.x & (kWave - 1)) == 0) red[threadIdx.x / kWave] = v;
    wait_lds_writes();
    hold_value(v);
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int i = 1; i < WAVES; ++i) v = v > red[i] ? v : red[i];
  }
  return v;
}

// Weights of V consecutive columns, from column e.
template <int V>
__device__ __forceinline__ void load_weights(const void* w, bool w_bf16, int64_t e, float* v) {
  if (!w) {
#pragma unroll
    for (int k = 0; k < V; ++k) v[k] = 1.0f;
  } else if (w_bf16) {
    const uint2* p = reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(w) + e);
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
      const uint2 u = p[i];
      v[4 * i] = bf16_low(u.x);
      v[4 * i + 1] = bf16_high(u.x);
      v[4 * i + 2] = bf16_low(u.y);
      v[4 * i + 3] = bf16_high(u.y);
    }
  } else {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(w) + e);
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
      const float4 u = p[i];
      v[4 * i] = u.x;
      v[4 * i + 1] = u.y;
      v[4 * i + 2] = u.z;
      v[4 * i + 3] = u.w;
    }
  }
}
__device__ __forceinline__ float load_weight(const void* w, bool w_bf16, int64_t e) {
  if (!w) return 1.0f;
  return w_bf16 ? bf16_low(static_cast<const uint16_t*>(w)[e]) : static_cast<const float*>(w)[e];
}

// A row over NT threads, C pieces of 16 bytes of x's type each: piece
// c * NT + t for thread t (WIDE: rows start 16-byte aligned and hold whole
// pieces).  Otherwise thread t holds elements i * NT + t, one load each.
// Q8: threads take their pieces in label order (lanes.h), so that the
// rotation's cross-lane stages are plain exchanges.
template <bool BF16, int NT, int C, bool WIDE, bool Q8>
__global__ void __launch_bounds__(NT < 256 ? 256 : NT)
norm_kernel(NormArgs a) {
  constexpr int V = Piece<BF16>::kElems, EB = Piece<BF16>::kBytes, N = C * V;
  constexpr int kTeams = NT < 256 ? 256 / NT : 1, kWaves = NT / kWave;
  __shared__ float red_f[kWaves];
  __shared__ uint32_t red_u[kWaves];
  const int t = threadIdx.x % NT;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kTeams + threadIdx.x / NT;
  if (kTeams > 1 && row >= a.rows) return;  // whole waves; one team per block has no such row
  const int label = lane_label(t & (kWave - 1));
  const int pos = Q8 ? (t & ~(kWave - 1)) | label : t;
  const int cols = static_cast<int>(a.cols);
  const int64_t first = row * a.cols;
  const uint8_t* const x = a.x + first * EB;
  const uint8_t* const r = a.residual ? a.residual + first * EB : nullptr;
  uint8_t* const sum = a.sum ? a.sum + first * EB : nullptr;

  float h[N];
  float ss = 0.0f;
  if constexpr (WIDE) {
    const int np = cols / V;
    uint4 xr[C], rr[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int p = c * NT + pos, pc = p < np ? p : 0;
      xr[c] = reinterpret_cast<const uint4*>(x)[pc];
    }
    if (r) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int p = c * NT + pos, pc = p < np ? p : 0;
        rr[c] = reinterpret_cast<const uint4*>(r)[pc];
      }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int p = c * NT + pos;
      unpack_piece<BF16>(xr[c], h + c * V);
      if (r) {
        float o[V];
        unpack_piece<BF16>(rr[c], o);
#pragma unroll
        for (int k = 0; k < V; ++k) h[c * V + k] += o[k];
      }
      if (p >= np) {
#pragma unroll
        for (int k = 0; k < V; ++k) h[c * V + k] = 0.0f;
      }
#pragma unroll
      for (int k = 0; k < V; ++k) ss = __builtin_fmaf(h[c * V + k], h[c * V + k], ss);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = i * NT + t, ec = e < cols ? e : 0;
      h[i] = load_elem<BF16>(x, ec);
      if (r) h[i] += load_elem<BF16>(r, ec);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (i * NT + t >= cols) h[i] = 0.0f;
      ss = __builtin_fmaf(h[i], h[i], ss);
    }
  }
  // x and residual are read: sum may be either of them.
  if (sum) {
    if constexpr (WIDE) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int p = c * NT + pos;
        if (p < cols / V) reinterpret_cast<uint4*>(sum)[p] = pack_piece<BF16>(h + c * V);
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i * NT + t < cols) store_elem<BF16>(sum, i * NT + t, h[i]);
    }
  }
  ss = block_sum<kWaves>(ss, red_f);
  const float rs = rsqrtf(ss / static_cast<float>(cols) + a.eps);

  if constexpr (!Q8) {
    if constexpr (WIDE) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int p = c * NT + pos;
        if (p >= cols / V) continue;
        float w[V], y[V];
        load_weights<V>(a.weight, a.w_bf16, static_cast<int64_t>(p) * V, w);
#pragma unroll
        for (int k = 0; k < V; ++k) y[k] = h[c * V + k] * rs * w[k];
        if (a.out_bf16) {
          uint32_t u[V / 2];
#pragma unroll
          for (int k = 0; k < V / 2; ++k) u[k] = pack_bf16(y[2 * k], y[2 * k + 1]);
          uint2* o = reinterpret_cast<uint2*>(a.out + first * 2) + static_cast<int64_t>(p) * (V / 4);
          if constexpr (V == 8)
            *reinterpret_cast<uint4*>(o) = make_uint4(u[0], u[1], u[V / 2 - 2], u[V / 2 - 1]);
          else
            *o = make_uint2(u[0], u[1]);
        } else {
          float4* o = reinterpret_cast<float4*>(a.out + first * 4) + static_cast<int64_t>(p) * (V / 4);
#pragma unroll
          for (int k = 0; k < V / 4; ++k) o[k] = make_float4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int e = i * NT + t;
        if (e >= cols) continue;
        const float y = h[i] * rs * load_weight(a.weight, a.w_bf16, e);
        if (a.out_bf16)
          store_elem<true>(a.out, first + e, y);
        else
          store_elem<false>(a.out, first + e, y);
      }
    }
  } else {
    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int p = c * NT + pos, pc = p < cols / V ? p : 0;
      float w[V];
      load_weights<V>(a.weight, a.w_bf16, static_cast<int64_t>(pc) * V, w);
      float y[V];
#pragma unroll
      for (int k = 0; k < V; ++k) y[k] = h[c * V + k] * rs * w[k];
      lane_butterfly(y);
      label_butterfly(y, label, a.labels);  // groups are whole runs of lanes: past the row they are zero or absent
#pragma unroll
      for (int k = 0; k < V; ++k) {
        h[c * V + k] = y[k];
        const uint32_t m = __builtin_bit_cast(uint32_t, y[k]) & 0x7FFFFFFFu;
        if (p < cols / V) top = top > m ? top : m;
      }
    }
    // As bit patterns: a NaN is above infinity, which is above every number.
    top = block_max<kWaves>(top, red_u);
    const float amax = __builtin_bit_cast(float, top);
    const bool finite = top < 0x7F800000u;
    // Below 2^-118 the reciprocal would leave float32: such a row is zero.
    const float inv = finite && amax >= 0x1.0p-118f ? 127.0f / amax : 0.0f;
    const float signed_inv = label_sign(label, a.labels) * inv;
    if (t == 0) a.scale[row] = !finite ? __builtin_nanf("") : inv == 0.0f ? 0.0f : amax * a.unit;
    int8_t* const q = a.q + first;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int p = c * NT + pos;
      if (p >= cols / V) continue;
      // fma(v, inv, 1.5 * 2^23) rounds v * inv to a whole number once; its
      // two's-complement byte is the sum's lowest (|v * inv| <= 127).
      uint32_t b[V];
#pragma unroll
      for (int k = 0; k < V; ++k)
        b[k] = inv == 0.0f ? 0u : __builtin_bit_cast(uint32_t, __builtin_fmaf(h[c * V + k], signed_inv, 12582912.0f));
      uint32_t u[V / 4];
#pragma unroll
      for (int k = 0; k < V / 4; ++k) {
        const uint32_t lo = __builtin_amdgcn_perm(b[4 * k + 1], b[4 * k], 0x0C0C0400u);
        const uint32_t hi = __builtin_amdgcn_perm(b[4 * k + 3], b[4 * k + 2], 0x04000C0Cu);
        u[k] = lo | hi;
      }
      if constexpr (V == 8)
        reinterpret_cast<uint2*>(q)[p] = make_uint2(u[0], u[V / 4 - 1]);
      else
        reinterpret_cast<uint32_t*>(q)[p] = u[0];
    }
  }
}

// Gradient.  A block takes rows blockIdx.x * teams + team, then every
// gridDim.x * teams-th; its share of dw stays in registers until its last
// row and goes to part[blockIdx.x], to be added in block order by
// weight_grad_kernel.  The next row's loads are issued before this row's
// reductions, which are the only waits.
template <bool BF16, int NT, int C, bool WIDE>
__global__ void __launch_bounds__(NT < 256 ? 256 : NT)
norm_grad_kernel(NormGradArgs a) {
  constexpr int V = Piece<BF16>::kElems, EB = Piece<BF16>::kBytes, N = C * V;
  constexpr int kTeams = NT < 256 ? 256 / NT : 1, kWaves = NT / kWave;
  constexpr int R = WIDE ? C : N;  // loads of one array per row
  typedef typename std::conditional<WIDE, uint4, uint32_t>::type Raw;
  __shared__ float red[2][2 * kWaves];
  __shared__ float team_dw[kTeams > 1 ? kTeams * NT * N : 1];
  const int t = threadIdx.x % NT, team = threadIdx.x / NT;
  const int cols = static_cast<int>(a.cols), np = cols / V;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kTeams;

  constexpr int M = WIDE ? V : 1;  // elements of one load
  float w[N], dw[N];
#pragma unroll
  for (int i = 0; i < N; ++i) dw[i] = 0.0f;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int p = i * NT + t;
    if constexpr (WIDE)
      load_weights<V>(a.weight, a.w_bf16, static_cast<int64_t>(p < np ? p : 0) * V, w + i * V);
    else
      w[i] = load_weight(a.weight, a.w_bf16, p < cols ? p : 0);
  }

  auto load = [&](const uint8_t* base, int64_t row, Raw (&v)[R]) __attribute__((always_inline)) {
    const uint8_t* p0 = base + row * a.cols * EB;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if constexpr (WIDE) {
        const int p = i * NT + t;
        v[i] = reinterpret_cast<const uint4*>(p0)[p < np ? p : 0];
      } else {
        const int e = i * NT + t < cols ? i * NT + t : 0;
        if constexpr (BF16)
          v[i] = reinterpret_cast<const uint16_t*>(p0)[e];
        else
          v[i] = reinterpret_cast<const uint32_t*>(p0)[e];
      }
    }
  };
  auto value = [](const Raw (&v)[R], int i) __attribute__((always_inline)) -> float {
    if constexpr (WIDE) {
      const uint4& p = v[i / V];
      const int k = i % V, d = BF16 ? k / 2 : k;
      const uint32_t u = d == 0 ? p.x : d == 1 ? p.y : d == 2 ? p.z : p.w;
      if constexpr (BF16)
        return k & 1 ? bf16_high(u) : bf16_low(u);
      else
        return __builtin_bit_cast(float, u);
    } else {
      if constexpr (BF16)
        return bf16_low(v[i]);
      else
        return __builtin_bit_cast(float, v[i]);
    }
  };
  auto inside = [&](int i) __attribute__((always_inline)) {
    return WIDE ? (i / V) * NT + t < np : i * NT + t < cols;
  };

  Raw h[R], dy[R], ds[R];
  int64_t row = static_cast<int64_t>(blockIdx.x) * kTeams + team;
  int turn = 0;
  if (row < a.rows) {
    load(a.sum, row, h);
    load(a.dout, row, dy);
    if (a.dsum) load(a.dsum, row, ds);
  }
  while (row < a.rows) {
    const int64_t next = row + stride;
    Raw h2[R], dy2[R], ds2[R];
    if (next < a.rows) {
      load(a.sum, next, h2);
      load(a.dout, next, dy2);
      if (a.dsum) load(a.dsum, next, ds2);
    }
    float ss = 0.0f, dot = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float hv = inside(i) ? value(h, i) : 0.0f;
      const float u = w[i] * value(dy, i);
      ss = __builtin_fmaf(hv, hv, ss);
      dot = inside(i) ? __builtin_fmaf(u, hv, dot) : dot;
    }
    ss = wave_sum(ss);
    dot = wave_sum(dot);
    if constexpr (kWaves > 1) {
      float* const slot = red[turn];  // two slots in turn: one barrier per row
      if ((threadIdx.x & (kWave - 1)) == 0) {
        slot[threadIdx.x / kWave] = ss;
        slot[kWaves + threadIdx.x / kWave] = dot;
      }
      wait_lds_writes();
      hold_values(ss, dot);
      __syncthreads();
      ss = slot[0];
      dot = slot[kWaves];
#pragma unroll
      for (int i = 1; i < kWaves; ++i) {
        ss += slot[i];
        dot += slot[kWaves + i];
      }
      turn ^= 1;
    }
    const float n = static_cast<float>(cols);
    const float r = rsqrtf(ss / n + a.eps);
    const float k = r * (dot / n);
    uint8_t* const out = a.dx + row * a.cols * EB;
#pragma unroll
    for (int l = 0; l < R; ++l) {
      const int p = l * NT + t;
      float d[M];
#pragma unroll
      for (int j = 0; j < M; ++j) {
        const int i = l * M + j;
        const float hn = value(h, i) * r, g = value(dy, i);
        d[j] = r * __builtin_fmaf(-hn, k, w[i] * g);
        if (a.dsum) d[j] += value(ds, i);
        if (inside(i)) dw[i] = __builtin_fmaf(g, hn, dw[i]);
      }
      if constexpr (WIDE) {
        if (p < np) reinterpret_cast<uint4*>(out)[p] = pack_piece<BF16>(d);
      } else {
        if (p < cols) store_elem<BF16>(out, p, d[0]);
      }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      h[i] = h2[i];
      dy[i] = dy2[i];
      ds[i] = ds2[i];
    }
    row = next;
  }

  if (!a.part) return;
  float* const part = a.part + blockIdx.x * a.cols;
  auto column = [&](int i, int tt) { return WIDE ? ((i / V) * NT + tt) * V + i % V : i * NT + tt; };
  if constexpr (kTeams > 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) team_dw[(team * N + i) * NT + t] = dw[i];
    wait_lds_writes();
#pragma unroll
    for (int i = 0; i < N; ++i) hold_value(dw[i]);
    __syncthreads();
    // Team k adds every kTeams-th of the N values over the teams, in order.
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (i % kTeams != team) continue;
      float s = team_dw[i * NT + t];
#pragma unroll
      for (int g = 1; g < kTeams; ++g) s += team_dw[(g * N + i) * NT + t];
      if (column(i, t) < cols) part[column(i, t)] = s;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (column(i, t) < cols) part[column(i, t)] = dw[i];
  }
}

// Gradient of wide rows.  Such a row does not fit the registers beside its
// share of dw: the block reads it twice (the second time from the L2, a row is
// at most 128 KiB) and keeps dw in LDS, each column with the thread that owns
// it.
constexpr int kWideThreads = 1024;
template <bool BF16, bool WIDE, int COLS>
__global__ void __launch_bounds__(kWideThreads)
norm_grad_wide_kernel(NormGradArgs a) {
  constexpr int V = WIDE ? Piece<BF16>::kElems : 1, EB = Piece<BF16>::kBytes, kWaves = kWideThreads / kWave;
  __shared__ float dw[COLS];
  __shared__ float red[2][2 * kWaves];
  const int t = threadIdx.x, np = static_cast<int>(a.cols) / V;
  auto load = [](const uint8_t* p, int i, float* v) __attribute__((always_inline)) {
    if constexpr (WIDE)
      unpack_piece<BF16>(reinterpret_cast<const uint4*>(p)[i], v);
    else
      v[0] = load_elem<BF16>(p, i);
  };
  auto weights = [&](int i, float* v) __attribute__((always_inline)) {
    if constexpr (WIDE)
      load_weights<V>(a.weight, a.w_bf16, static_cast<int64_t>(i) * V, v);
    else
      v[0] = load_weight(a.weight, a.w_bf16, i);
  };
  const float zero = 0.0f;
  for (int i = t; i < np; i += kWideThreads)
    for (int j = 0; j < V; ++j) dw[i * V + j] = zero;
  wait_lds_writes();
  hold_value(zero);
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const int64_t first = row * a.cols * EB;
    float ss = 0.0f, dot = 0.0f;
#pragma unroll 2
    for (int i = t; i < np; i += kWideThreads) {
      float h[V], g[V], w[V];
      load(a.sum + first, i, h);
      load(a.dout + first, i, g);
      weights(i, w);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        ss = __builtin_fmaf(h[j], h[j], ss);
        dot = __builtin_fmaf(w[j] * g[j], h[j], dot);
      }
    }
    ss = wave_sum(ss);
    dot = wave_sum(dot);
    float* const slot = red[turn];
    if ((t & (kWave - 1)) == 0) {
      slot[t / kWave] = ss;
      slot[kWaves + t / kWave] = dot;
    }
    wait_lds_writes();
    hold_values(ss, dot);
    __syncthreads();
    ss = slot[0];
    dot = slot[kWaves];
#pragma unroll
    for (int i = 1; i < kWaves; ++i) {
      ss += slot[i];
      dot += slot[kWaves + i];
    }
    turn ^= 1;
    const float n = static_cast<float>(a.cols);
    const float r = rsqrtf(ss / n + a.eps);
    const float k = r * (dot / n);
    for (int i = t; i < np; i += kWideThreads) {
      float h[V], g[V], w[V], d[V], s[V];
      load(a.sum + first, i, h);
      load(a.dout + first, i, g);
      weights(i, w);
      if (a.dsum) load(a.dsum + first, i, d);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float hn = h[j] * r, v = r * __builtin_fmaf(-hn, k, w[j] * g[j]);
        d[j] = a.dsum ? v + d[j] : v;
        s[j] = __builtin_fmaf(g[j], hn, dw[i * V + j]);
      }
      // dx may be dsum: this thread has read its own columns.
      if constexpr (WIDE)
        reinterpret_cast<uint4*>(a.dx + first)[i] = pack_piece<BF16>(d);
      else
        store_elem<BF16>(a.dx + first, i, d[0]);
#pragma unroll
      for (int j = 0; j < V; ++j) dw[i * V + j] = s[j];
      wait_lds_writes();
#pragma unroll
      for (int j = 0; j < V; ++j) hold_value(s[j]);
    }
  }
  if (!a.part) return;
  for (int i = t; i < np; i += kWideThreads)
    for (int j = 0; j < V; ++j) a.part[blockIdx.x * a.cols + i * V + j] = dw[i * V + j];
}

// dw[c] = sum over the blocks' shares, in a fixed order: 16 waves take every
// 16th share of 64 columns, their sums are added in wave order.
constexpr int kSumWaves = 16;
__global__ void __launch_bounds__(kSumWaves* kWave)
weight_grad_kernel(const float* __restrict__ part, int blocks, int64_t cols, float* __restrict__ dw) {
  __shared__ float s[kSumWaves][kWave];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kWave + lane, cc = c < cols ? c : cols - 1;
  float v = 0.0f;
#pragma unroll 8
  for (int b = wave; b < blocks; b += kSumWaves) v += part[b * cols + cc];
  s[wave][lane] = v;
  wait_lds_writes();
  hold_value(v);
  __syncthreads();
  if (wave == 0 && c < cols) {
    float t = s[0][lane];
#pragma unroll
    for (int i = 1; i < kSumWaves; ++i) t += s[i][lane];
    dw[c] = t;
  }
}

template <bool BF16, int NT, int C>
hipError_t launch_norm_at(NormArgs a, hipStream_t s) {
  constexpr int teams = NT < 256 ? 256 / NT : 1, threads = NT * teams;
  const bool wide = a.cols % Piece<BF16>::kElems == 0;
  for (int64_t left = a.rows; left > 0; left -= a.rows) {
    a.rows = left < most_blocks(threads) * teams ? left : most_blocks(threads) * teams;
    const dim3 grid(static_cast<uint32_t>((a.rows + teams - 1) / teams)), block(threads);
    if (a.q)
      norm_kernel<BF16, NT, C, true, true><<<grid, block, 0, s>>>(a);
    else if (wide)
      norm_kernel<BF16, NT, C, true, false><<<grid, block, 0, s>>>(a);
    else
      norm_kernel<BF16, NT, C, false, false><<<grid, block, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t done = a.rows * a.cols, bytes = done * Piece<BF16>::kBytes;
    a.x += bytes;
    if (a.residual) a.residual += bytes;
    if (a.sum) a.sum += bytes;
    if (a.q) {
      a.q += done;
      a.scale += a.rows;
    } else {
      a.out += done * (a.out_bf16 ? 2 : 4);
    }
  }
  return hipSuccess;
}

template <bool BF16, bool WIDE, int NT, int C>
hipError_t launch_norm_grad_at(const NormGradArgs& a, int blocks, hipStream_t s) {
  norm_grad_kernel<BF16, NT, C, WIDE><<<dim3(blocks), dim3(NT < 256 ? 256 : NT), 0, s>>>(a);
  return hipGetLastError();
}

template <bool BF16, bool WIDE>
hipError_t launch_norm_grad_wide(const NormGradArgs& a, int blocks, hipStream_t s) {
  const dim3 grid(blocks), block(kWideThreads);
  if (a.cols <= kNormMaxCols / 2)
    norm_grad_wide_kernel<BF16, WIDE, kNormMaxCols / 2><<<grid, block, 0, s>>>(a);
  else
    norm_grad_wide_kernel<BF16, WIDE, kNormMaxCols><<<grid, block, 0, s>>>(a);
  return hipGetLastError();
}

// The row's pieces of 16 bytes decide its team: one wave (no barrier) up to 64
// pieces, 4 waves up to 1024, then 16.  From 65 to 128 pieces one wave is the
// faster one with many rows: bf16 rows of 1024, one wave and four, 512 rows
// 3.2 and 3.0 us, 4096 rows 7.2 and 6.2, 8192 rows 10.6 and 11.8; to 8 bits,
// where each lane does more, 512 rows 3.8 and 3.2, 2048 rows 4.8 and 5.8, 4096
// rows 6.6 and 9.2.  From 513 to 1024 pieces 16 waves are with few: rows of
// 8192, 4 waves and 16, one row 2.9 and 2.0 us (to 8 bits 4.3 and 2.9), 512
// rows 6.4 and 6.6 (7.8 and 6.7), 1024 rows 10.9 and 12.0 (12.2 and 12.7).
template <bool BF16>
hipError_t launch_norm_for(const NormArgs& a, hipStream_t s) {
  const int64_t np = (a.cols + Piece<BF16>::kElems - 1) / Piece<BF16>::kElems, cus = device_cu_count();
  if (np <= 64) return launch_norm_at<BF16, 64, 1>(a, s);
  if (np <= 128 && a.rows >= (a.q ? 8 : 32) * cus) return launch_norm_at<BF16, 64, 2>(a, s);
  if (np <= 256) return launch_norm_at<BF16, 256, 1>(a, s);
  if (np <= 512) return launch_norm_at<BF16, 256, 2>(a, s);
  if (np <= 1024 && a.rows <= 2 * cus) return launch_norm_at<BF16, 1024, 1>(a, s);
  if (np <= 1024) return launch_norm_at<BF16, 256, 4>(a, s);
  if (np <= 2048) return launch_norm_at<BF16, 1024, 2>(a, s);
  if (np <= 4096) return launch_norm_at<BF16, 1024, 4>(a, s);
  if constexpr (!BF16) return launch_norm_at<BF16, 1024, 8>(a, s);
  return hipErrorInvalidValue;
}

// Rows that one wave takes, 4 of them to a block; others take the block.
bool norm_grad_one_wave(int64_t cols, bool bf16) {
  const int64_t v = bf16 ? 8 : 4, np = (cols + v - 1) / v;
  return np <= 64 || (np <= 128 && (cols % v == 0 || !bf16));
}

// Up to 8 elements per lane the row, the next one and dw stay in registers
// (one element per load) and up to 16 in whole pieces.  Rows beyond that go to
// the wide kernel: bf16, 8192 columns, 256 rows 7.1 us (11.1 from registers,
// 32 elements per lane), 4096 rows 67.3 (73.3); 4001 columns, 4096 rows 38.5
// (81.0, 16 single elements).  So do up to four rows per CU of 16 elements per
// lane: bf16, 4096 columns, 300 rows 5.9 us (8.0), 1024 rows 10.8 (11.8), 4096
// rows 34.9 (26.6); float32 7.0 (7.0), 13.4 (14.5), 48.2 (44.2).
template <bool BF16, bool WIDE>
hipError_t launch_norm_grad_for(const NormGradArgs& a, int blocks, hipStream_t s) {
  const int64_t np = (a.cols + Piece<BF16>::kElems - 1) / Piece<BF16>::kElems;
  if (np <= 64) return launch_norm_grad_at<BF16, WIDE, 64, 1>(a, blocks, s);
  if constexpr (WIDE || !BF16) {
    if (np <= 128) return launch_norm_grad_at<BF16, WIDE, 64, 2>(a, blocks, s);
  }
  if (np <= 256) return launch_norm_grad_at<BF16, WIDE, 256, 1>(a, blocks, s);
  if constexpr (!BF16) {
    if (np <= 512) return launch_norm_grad_at<BF16, WIDE, 256, 2>(a, blocks, s);
  }
  if constexpr (WIDE) {
    constexpr int kPieces = BF16 ? 2 : 4;
    if (np <= 256 * kPieces && a.rows > 4 * static_cast<int64_t>(device_cu_count()))
      return launch_norm_grad_at<BF16, WIDE, 256, kPieces>(a, blocks, s);
  }
  return launch_norm_grad_wide<BF16, WIDE>(a, blocks, s);
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, bool bf16, hipStream_t s) {
  return bf16 ? launch_norm_for<true>(a, s) : launch_norm_for<false>(a, s);
}

// Blocks of the gradient: as many as there are rows, up to two per CU of the
// MI355X; each leaves one share of dw.
int norm_grad_blocks(int64_t rows, int64_t cols, bool bf16) {
  const int64_t teams = norm_grad_one_wave(cols, bf16) ? 4 : 1, want = (rows + teams - 1) / teams;
  return static_cast<int>(want < kNormGradBlocks ? want : kNormGradBlocks);
}

hipError_t launch_norm_grad(NormGradArgs a, bool bf16, float* dweight, float* ws, hipStream_t s) {
  const int blocks = norm_grad_blocks(a.rows, a.cols, bf16);
  a.part = !dweight ? nullptr : blocks == 1 ? dweight : ws;
  const bool wide = a.cols % (bf16 ? 8 : 4) == 0;
  const hipError_t e = bf16 ? (wide ? launch_norm_grad_for<true, true>(a, blocks, s) : launch_norm_grad_for<true, false>(a, blocks, s))
                            : (wide ? launch_norm_grad_for<false, true>(a, blocks, s) : launch_norm_grad_for<false, false>(a, blocks, s));
  if (e != hipSuccess || !dweight || blocks == 1) return e;
  weight_grad_kernel<<<dim3(static_cast<uint32_t>((a.cols + kWave - 1) / kWave)), dim3(kSumWaves * kWave), 0, s>>>(
      a.part, blocks, a.cols, dweight);
  return hipGetLastError();
}

}  // namespace cq
