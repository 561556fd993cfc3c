// Gradient of attention (attention.hip) with respect to queries, keys and
// values, from the forward's output and lse.  With x = scale q . k,
// P = exp(x - lse), D_i = sum_d dout_i out_i:
//   dv_j = sum_i P_ij dout_i,   dS_ij = P_ij (dout_i . v_j - D_i),
//   dq_i = scale sum_j dS_ij k_j,   dk_j = scale sum_i dS_ij q_i,
// keys' sums over all query heads of the group.
//
// Two kernels, one that owns rows of queries and walks over the keys, one that
// owns keys and walks over the rows: each forms the probabilities again, 7
// products where 5 would do, but every sum then has one owner and a fixed
// order.  (One kernel would have to add dq with atomics, or write a share of
// dq per tile of keys to memory.)  P and dS are rounded to bf16 for bf16
// inputs, half a step of each term.
#include "attention.h"

namespace cq {
namespace {

constexpr int kWaves = 4;
constexpr int kBlockRows = kWaves * kRows;
constexpr int kTileKeys = 64;

// The workspace: log of the sum in powers of two, then D, each [q_heads][rows_q].
__device__ __forceinline__ float* log_sums(const AttnArgs& a, int64_t head) { return a.ws + head * a.seqs.rows_q; }
__device__ __forceinline__ float* dots(const AttnArgs& a, int64_t head) {
  return a.ws + (a.q_heads + head) * a.seqs.rows_q;
}

// dq, and D and the log sums for the second kernel.  The walk of
// attention_kernel, with v read by rows and k by columns.
template <bool BF16, int DP>
__global__ void __launch_bounds__(kWaves * kWave, BF16 ? 2 : 1) attention_dq_kernel(AttnArgs a, int64_t tiles) {
  typedef Tile<BF16, DP, kTileKeys> T;
  constexpr int kElem = T::kElem, kSubs = kTileKeys / 32, kDepth = DP / 16, kDt = DP / 32;
  __shared__ __attribute__((aligned(16))) uint8_t k_tile0[T::kBytes], k_tile1[T::kBytes], v_tile0[T::kBytes], v_tile1[T::kBytes];
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), half = lane >> 5;
  const int group = a.q_heads / a.kv_heads;
  const int kv_head = static_cast<int>(blockIdx.x % a.kv_heads);
  SeqRows seq;
  int64_t tile;
  if (!find_tile(a.seqs, tiles - 1 - blockIdx.x / a.kv_heads,
                 [&](const SeqRows& s) { return (s.nq * group + kBlockRows - 1) / kBlockRows; }, &seq, &tile))
    return;
  const int64_t rows = seq.nq * group, r0 = tile * kBlockRows + wave * kRows;
  const Row row = row_of(r0 + (lane & 31), rows, group);
  const int64_t block_last = row_of(min(tile * kBlockRows + kBlockRows, rows) - 1, rows, group).query;
  const int64_t wave_last = row_of(min(r0 + kRows, rows) - 1, rows, group).query;
  const int64_t block_keys = keys_seen(seq, block_last, a.causal);
  const int64_t wave_keys = r0 < rows ? keys_seen(seq, wave_last, a.causal) : 0;
  const int64_t all_see = r0 < rows ? keys_seen(seq, row_of(r0, rows, group).query, a.causal) : 0;
  const int64_t seen = row.exists ? keys_seen(seq, row.query, a.causal) : 0;
  const int64_t at = seq.q0 + row.query, head = static_cast<int64_t>(kv_head) * group + row.head;

  Operand<BF16> q[kDepth], dout[kDepth];
  load_row_operands<BF16, DP>(row.exists ? row_data(a.q, at, head, kElem) : nullptr, a.head_dim, half, q);
  load_row_operands<BF16, DP>(row.exists ? row_data(a.dout, at, head, kElem) : nullptr, a.head_dim, half, dout);
  float dot = 0.0f, log_sum = INFINITY;  // a row without keys, or none: P = 0
  {
    Operand<BF16> out[kDepth];
    load_row_operands<BF16, DP>(row.exists ? row_data(a.out, at, head, kElem) : nullptr, a.head_dim, half, out);
#pragma unroll
    for (int kk = 0; kk < kDepth; ++kk)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        dot = __builtin_fmaf(static_cast<float>(dout[kk][j]), static_cast<float>(out[kk][j]), dot);
    float x, y;
    both_halves(dot, &x, &y);
    dot = x + y;
    if (row.exists) {
      const float lse = a.lse[at * a.q_heads + head];
      log_sum = lse == -INFINITY ? INFINITY : lse * kLog2e;
      if (half == 0) {
        log_sums(a, head)[at] = log_sum;
        dots(a, head)[at] = dot;
      }
    }
  }

  const TileLoader<BF16, DP, kTileKeys, kWaves> k_load(wave, lane, a.k.row, a.head_dim), v_load(wave, lane, a.v.row, a.head_dim);
  const RowOperand<BF16, DP> by_row(lane);
  const ColumnOperand<BF16, DP> by_column(lane);
  const uint8_t* const k0 = row_data(a.k, seq.k0, kv_head, kElem);
  const uint8_t* const v0 = row_data(a.v, seq.k0, kv_head, kElem);
  const float factor = a.scale * kLog2e;

  f32_x16 dq[kDt];
#pragma unroll
  for (int dt = 0; dt < kDt; ++dt)
#pragma unroll
    for (int r = 0; r < 16; ++r) dq[dt][r] = 0.0f;

  const int64_t n_tiles = (block_keys + kTileKeys - 1) / kTileKeys;
  auto issue = [&](int64_t t, uint8_t* kt, uint8_t* vt) __attribute__((always_inline)) {
    const int64_t key = t * kTileKeys;
    k_load.issue(k0 + key * a.k.row * kElem, seq.nk - key, kt);
    v_load.issue(v0 + key * a.v.row * kElem, seq.nk - key, vt);
  };
  auto compute = [&](int64_t t, const uint8_t* kt, const uint8_t* vt) __attribute__((always_inline)) {
    const int64_t key = t * kTileKeys;
    if (key >= wave_keys) return;
    const int left = static_cast<int>(min(seen - key, int64_t(kTileKeys))) - 4 * half;
    const bool masked = key + kTileKeys > all_see;
#pragma unroll
    for (int sub = 0; sub < kSubs; ++sub) {
      f32_x16 s, dp;
#pragma unroll
      for (int r = 0; r < 16; ++r) s[r] = dp[r] = 0.0f;
#pragma unroll
      for (int kk = 0; kk < kDepth; ++kk) {
        multiply<BF16>(s, by_row.load(kt, sub, kk), q[kk]);
        multiply<BF16>(dp, by_row.load(vt, sub, kk), dout[kk]);
      }
#pragma unroll
      for (int r = 0; r < 16; ++r) s[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r], factor, -log_sum)) * (dp[r] - dot);
      if (masked) {
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (32 * sub + result_row(r) >= left) s[r] = 0.0f;
      }
#pragma unroll
      for (int step = 0; step < 2; ++step) {
        const Operand<BF16> ds = result_operand<BF16>(s, step);
#pragma unroll
        for (int dt = 0; dt < kDt; ++dt) multiply<BF16>(dq[dt], by_column.load(kt, 2 * sub + step, dt), ds);
      }
    }
  };

  if (n_tiles > 0) issue(0, k_tile0, v_tile0);
  for (int64_t t = 0; t < n_tiles; t += 2) {
    wait_loads<0>();
    __syncthreads();
    if (t + 1 < n_tiles) issue(t + 1, k_tile1, v_tile1);
    compute(t, k_tile0, v_tile0);
    if (t + 1 >= n_tiles) break;
    wait_loads<0>();
    __syncthreads();
    if (t + 2 < n_tiles) issue(t + 2, k_tile0, v_tile0);
    compute(t + 1, k_tile1, v_tile1);
  }
  store_columns<BF16, DP>(dq, a.scale, row.exists ? row_data(a.dq, at, head, kElem) : nullptr, a.head_dim, half);
}

// dk and dv of 128 keys, 32 per wave, over the rows of every head of the group
// in tiles of 64.  Scores are formed as q . k^T here: a lane holds 16 rows of
// one key, which is the operand of both sums over the rows.
constexpr int kTileRows = 64;

template <bool BF16, int DP>
__global__ void __launch_bounds__(kWaves * kWave, 1) attention_dkv_kernel(AttnArgs a) {
  typedef Tile<BF16, DP, kTileRows> T;
  constexpr int kElem = T::kElem, kSubs = kTileRows / 32, kDepth = DP / 16, kDt = DP / 32;
  __shared__ __attribute__((aligned(16))) uint8_t q_tile0[T::kBytes], q_tile1[T::kBytes], do_tile0[T::kBytes], do_tile1[T::kBytes];
  __shared__ __attribute__((aligned(16))) float stat0[2 * kTileRows], stat1[2 * kTileRows];  // log sums, D
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), half = lane >> 5;
  const int group = a.q_heads / a.kv_heads;
  const int kv_head = static_cast<int>(blockIdx.x % a.kv_heads);
  SeqRows seq;
  int64_t tile;
  if (!find_tile(a.seqs, blockIdx.x / a.kv_heads, [&](const SeqRows& s) { return (s.nk + kBlockRows - 1) / kBlockRows; }, &seq,
                 &tile))
    return;
  const int64_t key0 = tile * kBlockRows, wave_key = key0 + wave * kRows, key = wave_key + (lane & 31);
  const bool exists = key < seq.nk;
  // Row i sees keys up to i + ahead.
  const int64_t ahead = seq.nk - seq.nq;
  const int64_t first_row = a.causal ? cut(key0 - ahead, 0, seq.nq) : 0;  // the first that sees key0
  const int64_t first_tile = first_row / kTileRows, row_tiles = (seq.nq + kTileRows - 1) / kTileRows;
  const int64_t per_head = seq.nq > first_row ? row_tiles - first_tile : 0;

  Operand<BF16> k[kDepth], v[kDepth];
  load_row_operands<BF16, DP>(exists ? row_data(a.k, seq.k0 + key, kv_head, kElem) : nullptr, a.head_dim, half, k);
  load_row_operands<BF16, DP>(exists ? row_data(a.v, seq.k0 + key, kv_head, kElem) : nullptr, a.head_dim, half, v);
  const TileLoader<BF16, DP, kTileRows, kWaves> q_load(wave, lane, a.q.row, a.head_dim), do_load(wave, lane, a.dout.row, a.head_dim);
  const RowOperand<BF16, DP> by_row(lane);
  const ColumnOperand<BF16, DP> by_column(lane);
  const float factor = a.scale * kLog2e;

  f32_x16 dk[kDt], dv[kDt];
#pragma unroll
  for (int dt = 0; dt < kDt; ++dt)
#pragma unroll
    for (int r = 0; r < 16; ++r) dk[dt][r] = dv[dt][r] = 0.0f;

  // Turn u is tile first_tile + u % per_head of head u / per_head of the group; the loader is one turn ahead.
  const int64_t turns = per_head * group;
  int64_t load_tile = first_tile, load_head = static_cast<int64_t>(kv_head) * group, this_tile = first_tile;
  auto issue = [&](uint8_t* qt, uint8_t* dot, float* stat) __attribute__((always_inline)) {
    const int64_t i = load_tile * kTileRows, left = seq.nq - i;
    q_load.issue(row_data(a.q, seq.q0 + i, load_head, kElem), left, qt);
    do_load.issue(row_data(a.dout, seq.q0 + i, load_head, kElem), left, dot);
#if defined(__HIP_DEVICE_COMPILE__)
    if (wave < 2) {
      // Rows past the sequence read as zeros: P = 1 there, times dout = 0.
      float* const p = (wave ? dots(a, load_head) : log_sums(a, load_head)) + seq.q0 + i;
      const auto src = __builtin_amdgcn_make_buffer_rsrc(p, 0, static_cast<int>(min(left, int64_t(kTileRows)) * 4), 0x00020000);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (lds_void_ptr)(stat + wave * kTileRows), 4, lane * 4, 0, 0, 0);
    }
#endif
    if (++load_tile == row_tiles) {
      load_tile = first_tile;
      ++load_head;
    }
  };
  auto compute = [&](const uint8_t* qt, const uint8_t* dot, const float* stat) __attribute__((always_inline)) {
    const int64_t i0 = this_tile * kTileRows;
    if (++this_tile == row_tiles) this_tile = first_tile;
    if (wave_key >= seq.nk) return;
#pragma unroll
    for (int sub = 0; sub < kSubs; ++sub) {
      const int64_t i = i0 + 32 * sub;
      if (a.causal && i + 31 + ahead < wave_key) continue;  // no row of these sees a key of this wave
      f32_x16 s, dp;
#pragma unroll
      for (int r = 0; r < 16; ++r) s[r] = dp[r] = 0.0f;
#pragma unroll
      for (int kk = 0; kk < kDepth; ++kk) {
        multiply<BF16>(s, by_row.load(qt, sub, kk), k[kk]);
        multiply<BF16>(dp, by_row.load(dot, sub, kk), v[kk]);
      }
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const float4 ls = *reinterpret_cast<const float4*>(stat + 32 * sub + 8 * g + 4 * half);
        const float4 dd = *reinterpret_cast<const float4*>(stat + kTileRows + 32 * sub + 8 * g + 4 * half);
        const float l[4] = {ls.x, ls.y, ls.z, ls.w}, d[4] = {dd.x, dd.y, dd.z, dd.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = 4 * g + j;
          s[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r], factor, -l[j]));
          dp[r] = s[r] * (dp[r] - d[j]);
        }
      }
      if (a.causal && i + ahead < wave_key + 31) {
        const int see = static_cast<int>(cut(key - ahead - i, 0, 32)) - 4 * half;  // rows from here on see the key
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (result_row(r) < see) s[r] = dp[r] = 0.0f;
      }
#pragma unroll
      for (int step = 0; step < 2; ++step) {
        const Operand<BF16> p = result_operand<BF16>(s, step), ds = result_operand<BF16>(dp, step);
#pragma unroll
        for (int dt = 0; dt < kDt; ++dt) {
          multiply<BF16>(dv[dt], by_column.load(dot, 2 * sub + step, dt), p);
          multiply<BF16>(dk[dt], by_column.load(qt, 2 * sub + step, dt), ds);
        }
      }
    }
  };

  if (turns > 0) issue(q_tile0, do_tile0, stat0);
  for (int64_t u = 0; u < turns; u += 2) {
    wait_loads<0>();
    __syncthreads();
    if (u + 1 < turns) issue(q_tile1, do_tile1, stat1);
    compute(q_tile0, do_tile0, stat0);
    if (u + 1 >= turns) break;
    wait_loads<0>();
    __syncthreads();
    if (u + 2 < turns) issue(q_tile0, do_tile0, stat0);
    compute(q_tile1, do_tile1, stat1);
  }
  store_columns<BF16, DP>(dk, a.scale, exists ? row_data(a.dk, seq.k0 + key, kv_head, kElem) : nullptr, a.head_dim, half);
  store_columns<BF16, DP>(dv, 1.0f, exists ? row_data(a.dv, seq.k0 + key, kv_head, kElem) : nullptr, a.head_dim, half);
}

int64_t k_tiles(const AttnSeqs& s) {
  return tile_bound(s, s.k_starts ? -1 : s.rows_k / s.n_seq, s.rows_k, kBlockRows);
}

template <bool BF16, int DP>
hipError_t launch_at(const AttnArgs& a, hipStream_t stream) {
  const int64_t tiles = q_tiles(a.seqs, a.q_heads / a.kv_heads, kBlockRows);
  if (tiles)
    attention_dq_kernel<BF16, DP><<<dim3(static_cast<uint32_t>(tiles * a.kv_heads)), dim3(kWaves * kWave), 0, stream>>>(a, tiles);
  const int64_t kt = k_tiles(a.seqs);
  if (kt) attention_dkv_kernel<BF16, DP><<<dim3(static_cast<uint32_t>(kt * a.kv_heads)), dim3(kWaves * kWave), 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

int64_t attention_grad_workspace(const AttnSeqs& s, int q_heads, int kv_heads, int head_dim, bool bf16) {
  return 2 * s.rows_q * q_heads * 4;
}

int64_t attention_grad_blocks(const AttnSeqs& s, int q_heads, int kv_heads, int head_dim, bool bf16) {
  const int64_t q = q_tiles(s, q_heads / kv_heads, kBlockRows), k = k_tiles(s);
  return (q > k ? q : k) * kv_heads;
}

hipError_t launch_attention_grad(const AttnArgs& a, bool bf16, hipStream_t s) {
  if (bf16) return a.head_dim <= 64 ? launch_at<true, 64>(a, s) : launch_at<true, 128>(a, s);
  return a.head_dim <= 64 ? launch_at<false, 64>(a, s) : launch_at<false, 128>(a, s);
}

}  // namespace cq
