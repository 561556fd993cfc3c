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
// inputs, half a step of each term, and D is taken with the out that the forward
// stored, bf16's half step of each value: it is what a caller keeps of the forward,
// and D without it would take one more walk over the keys.  The error of dq and dk,
// relative to their root mean square: 0.0017 from their own rounding, 0.0024 with that of
// dS, 0.0025 with D's over 500 keys, 0.0029 over 64.
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
// attention_kernel, with v read by rows and k by columns.  8192 tokens in 3
// sequences, 32 heads of 128 over 8, bf16: 296 us, 0.96 PFLOP/s; the matrix cores
// are busy 54% of the cycles, the vector units 43%, shared memory's reads 28%.
template <bool BF16, int DP>
__global__ void __launch_bounds__(kWaves * kWave, BF16 ? 2 : 1) attention_dq_kernel(AttnArgs a) {
  typedef Tile<BF16, DP, kTileKeys> T;
  constexpr int kElem = T::kElem, kSubs = kTileKeys / 32, kDepth = DP / 16, kDt = DP / 32;
  __shared__ __attribute__((aligned(16))) uint8_t k_tile0[T::kBytes], k_tile1[T::kBytes], v_tile0[T::kBytes], v_tile1[T::kBytes];
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), half = lane >> 5;
  const int group = a.q_heads / a.kv_heads;
  const int kv_head = static_cast<int>(blockIdx.x % a.kv_heads);
  SeqRows seq;
  int64_t tile;
  if (!find_tile<true, !BF16>(a.seqs, blockIdx.x / a.kv_heads,
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
  [[maybe_unused]] const uint8_t* const k0 = row_data(a.k, seq.k0, kv_head, kElem);
  [[maybe_unused]] const uint8_t* const v0 = row_data(a.v, seq.k0, kv_head, kElem);
  const float factor = a.scale * kLog2e;

  f32_x16 dq[kDt];
#pragma unroll
  for (int dt = 0; dt < kDt; ++dt)
#pragma unroll
    for (int r = 0; r < 16; ++r) dq[dt][r] = 0.0f;

  const int64_t n_tiles = (block_keys + kTileKeys - 1) / kTileKeys;
  // The loads of a tile: begin(), then load(i) for each i < kLoads.  Spread over
  // the products of the tile before: in one stretch they wait for each other,
  // and the wave with them.
  constexpr int kLoads = 2 * TileLoader<BF16, DP, kTileKeys, kWaves>::kLoads;
  [[maybe_unused]] int keys_here = 0;  // of the tile being loaded; past the last: none
#if defined(__HIP_DEVICE_COMPILE__)
  __amdgpu_buffer_rsrc_t k_src, v_src;
#endif
  auto begin = [&](int64_t t) __attribute__((always_inline)) {
    const int64_t key = t * kTileKeys;
    keys_here = __builtin_amdgcn_readfirstlane(t < n_tiles ? static_cast<int>(min(seq.nk - key, int64_t(kTileKeys))) : 0);
#if defined(__HIP_DEVICE_COMPILE__)
    k_src = k_load.source(k0 + key * a.k.row * kElem, keys_here);
    v_src = v_load.source(v0 + key * a.v.row * kElem, keys_here);
#endif
  };
  auto load = [&](int i, uint8_t* kt, uint8_t* vt) __attribute__((always_inline)) {
#if defined(__HIP_DEVICE_COMPILE__)
    if (i < kLoads / 2)
      k_load.issue(k_src, i, keys_here, kt);
    else
      v_load.issue(v_src, i - kLoads / 2, keys_here, vt);
#endif
  };
  auto load_all = [&](uint8_t* kt, uint8_t* vt) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) load(i, kt, vt);
  };
  auto compute = [&](int64_t t, const uint8_t* kt, const uint8_t* vt, uint8_t* next_k, uint8_t* next_v) __attribute__((always_inline)) {
    const int64_t key = t * kTileKeys;
    begin(t + 1);
    if (key >= wave_keys) {
      load_all(next_k, next_v);
      return;
    }
    const int left = static_cast<int>(min(seen - key, int64_t(kTileKeys))) - 4 * half;
    const bool masked = key + kTileKeys > all_see;
#pragma unroll
    for (int sub = 0; sub < kSubs; ++sub) {
      f32_x16 s, dp;
#pragma unroll
      for (int r = 0; r < 16; ++r) s[r] = dp[r] = 0.0f;
      constexpr int kAhead = 4;  // operands read before their product
      auto operand = [&](int n) __attribute__((always_inline)) { return by_row.load(n & 1 ? vt : kt, sub, n >> 1); };
      Operand<BF16> rows_of[2 * kDepth];
#pragma unroll
      for (int n = 0; n < kAhead; ++n) rows_of[n] = operand(n);
#pragma unroll
      for (int n = 0; n < 2 * kDepth; ++n) {
        constexpr int kApart = kSubs * 2 * kDepth / kLoads;  // products between loads
        static_assert(kApart * kLoads == kSubs * 2 * kDepth, "loads at even distances");
        if ((sub * 2 * kDepth + n) % kApart == 0) load((sub * 2 * kDepth + n) / kApart, next_k, next_v);
        if (n + kAhead < 2 * kDepth) rows_of[n + kAhead] = operand(n + kAhead);
        if (n & 1)
          multiply<BF16>(dp, rows_of[n], dout[n >> 1]);
        else
          multiply<BF16>(s, rows_of[n], q[n >> 1]);
        if constexpr (BF16) pin();
      }
#pragma unroll
      for (int r = 0; r < 16; ++r) s[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r], factor, -log_sum)) * (dp[r] - dot);
      if (masked) {
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (32 * sub + result_row(r) >= left) s[r] = 0.0f;
      }
      Operand<BF16> columns[2 * kDt];
#pragma unroll
      for (int n = 0; n < kDt; ++n) columns[n] = by_column.load(kt, 2 * sub, n);
#pragma unroll
      for (int n = 0; n < 2 * kDt; ++n) {
        const Operand<BF16> ds = result_operand<BF16>(s, n / kDt);
        if (n < kDt) columns[n + kDt] = by_column.load(kt, 2 * sub + 1, n);
        multiply<BF16>(dq[n % kDt], columns[n], ds);
        if constexpr (BF16) pin();
      }
    }
  };

  if (n_tiles > 0) {
    begin(0);
    load_all(k_tile0, v_tile0);
  }
  for (int64_t t = 0; t < n_tiles; t += 2) {
    wait_loads<0>();
    __syncthreads();
    compute(t, k_tile0, v_tile0, k_tile1, v_tile1);
    if (t + 1 >= n_tiles) break;
    wait_loads<0>();
    __syncthreads();
    compute(t + 1, k_tile1, v_tile1, k_tile0, v_tile0);
  }
  wait_loads<0>();  // none is under way into memory that is given back

  store_columns<BF16, DP>(dq, a.scale, row.exists ? row_data(a.dq, at, head, kElem) : nullptr, a.head_dim, half);
}

// dk and dv of a block's keys, 32 per wave, over the rows of every head of the
// group in turns of 32.  Scores are formed as q . k^T here: a lane holds 16
// rows of one key, which is the operand of both sums over the rows.
//
// A wave needs 128 registers for dk and dv and 64 for its keys and values, so
// one wave has a SIMD to itself and nothing else fills its waits: the next
// turn's scores are formed while this turn's probabilities are (their
// instructions interleaved), and rows are loaded three turns ahead into a ring
// of four (in arrays of their own, as the compiler waits for all loads under way
// where it cannot tell their places apart).
//
// HEADS: streams of heads in a block.  The first keys of a long sequence are
// seen by all its rows, so one stream over all heads of the group makes a few
// blocks that outlast the others; two streams over half of the heads each, by
// two waves of 32 keys each, halve the longest block, and their sums meet in
// shared memory.  Whole gradients of bf16, two streams (one): one sequence of 4096
// tokens, 32 heads of 128 over 8, 486 us (634), 8 of 64 over 2, 246 (417); where blocks
// are many the order of their work alone is enough: 8192 tokens in 3 sequences,
// 32 heads of 128 over 8, 804 (818).
//
// 8192 tokens in 3 sequences, 32 heads of 128 over 8, bf16: 466 us, up to 526 on other
// cards, 0.72 to 0.81 PFLOP/s; the matrix cores are busy 44% of the cycles, the vector units 34%,
// waves wait 22%, and the last blocks end 10% after the average one.  Two
// waves per SIMD do not fit the registers (with part of v read from shared
// memory 705 us).
constexpr int kTurnRows = 32;

template <bool BF16, int DP, int HEADS>
__global__ void __launch_bounds__(kWaves * kWave, 1) attention_dkv_kernel(AttnArgs a) {
  typedef Tile<BF16, DP, kTurnRows> T;
  constexpr int kElem = T::kElem, kDepth = DP / 16, kDt = DP / 32, kKeyWaves = kWaves / HEADS, kBlockKeys = kKeyWaves * kRows;
  constexpr int kBytes = HEADS * T::kBytes, kStat = HEADS * 2 * kWave;
  __shared__ __attribute__((aligned(16))) uint8_t q0[kBytes], q1[kBytes], q2[kBytes], q3[kBytes];
  __shared__ __attribute__((aligned(16))) uint8_t do0[kBytes], do1[kBytes], do2[kBytes], do3[kBytes];
  __shared__ __attribute__((aligned(16))) float stat0[kStat], stat1[kStat], stat2[kStat], stat3[kStat];  // log sums, D
  const int lane = threadIdx.x & (kWave - 1), half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave) % kKeyWaves;    // along the keys
  const int stream = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave) / kKeyWaves;  // of heads
  const int group = a.q_heads / a.kv_heads;
  const int kv_head = static_cast<int>(blockIdx.x % a.kv_heads);
  SeqRows seq;
  int64_t tile;
  if (!find_tile<false, true>(a.seqs, blockIdx.x / a.kv_heads, [&](const SeqRows& s) { return (s.nk + kBlockKeys - 1) / kBlockKeys; }, &seq,
                 &tile))
    return;
  const int64_t key0 = tile * kBlockKeys, wave_key = key0 + wave * kRows, key = wave_key + (lane & 31);
  const bool exists = key < seq.nk;
  // Row i sees keys up to i + ahead.
  const int64_t ahead = seq.nk - seq.nq;
  const int64_t first_row = a.causal ? cut(key0 - ahead, 0, seq.nq) / kTurnRows * kTurnRows : 0;  // of the turn with the first that sees key0
  const int64_t per_head = (seq.nq - first_row + kTurnRows - 1) / kTurnRows;
  const int64_t turns = per_head * ((group + HEADS - 1) / HEADS);  // of the longest stream

  Operand<BF16> k[kDepth], v[kDepth];
  load_row_operands<BF16, DP>(exists ? row_data(a.k, seq.k0 + key, kv_head, kElem) : nullptr, a.head_dim, half, k);
  load_row_operands<BF16, DP>(exists ? row_data(a.v, seq.k0 + key, kv_head, kElem) : nullptr, a.head_dim, half, v);
  const TileLoader<BF16, DP, kTurnRows, kKeyWaves> q_load(wave, lane, a.q.row, a.head_dim), do_load(wave, lane, a.dout.row, a.head_dim);
  constexpr int kLoads = 2 * TileLoader<BF16, DP, kTurnRows, kKeyWaves>::kLoads;  // of a turn, without the statistics
  const RowOperand<BF16, DP> by_row(lane, stream * T::kBytes);
  const ColumnOperand<BF16, DP> by_column(lane, stream * T::kBytes);
  const float factor = a.scale * kLog2e;

  f32_x16 dk[kDt], dv[kDt];
#pragma unroll
  for (int dt = 0; dt < kDt; ++dt)
#pragma unroll
    for (int r = 0; r < 16; ++r) dk[dt][r] = dv[dt][r] = 0.0f;

  // A stream's turns: the rows from first_row on of heads stream, stream + HEADS, ... of the group.
  int head = stream, load_turn = 0;  // being loaded
  const int last_turn = static_cast<int>(per_head) - 1, last_rows = static_cast<int>(seq.nq - first_row - int64_t(last_turn) * kTurnRows);
  [[maybe_unused]] const uint8_t *q_at, *do_at;
  [[maybe_unused]] const float* stat_at;
  auto start_head = [&]() __attribute__((always_inline)) {
    const int64_t h = static_cast<int64_t>(kv_head) * group + (head < group ? head : 0);
    q_at = row_data(a.q, seq.q0 + first_row, h, kElem);
    do_at = row_data(a.dout, seq.q0 + first_row, h, kElem);
    stat_at = (wave ? dots(a, h) : log_sums(a, h)) + seq.q0 + first_row;
  };
  start_head();
  const int64_t q_turn = kTurnRows * a.q.row * kElem, do_turn = kTurnRows * a.dout.row * kElem;
  // The loads of a turn: begin(), then load(i) for each i < kLoads.  Spread over
  // a turn's products: in one stretch they wait for each other, and the wave with them.
  [[maybe_unused]] int rows_here = 0;  // of the turn being loaded; past the last head: none, zeros add nothing
#if defined(__HIP_DEVICE_COMPILE__)
  __amdgpu_buffer_rsrc_t q_src, do_src;
#endif
  auto begin = [&](float* stat) __attribute__((always_inline)) {
    rows_here = __builtin_amdgcn_readfirstlane(head >= group ? 0 : load_turn < last_turn ? kTurnRows : last_rows);
#if defined(__HIP_DEVICE_COMPILE__)
    q_src = q_load.source(q_at, rows_here);
    do_src = do_load.source(do_at, rows_here);
    if (wave < 2) {
      // Rows past the sequence read as zeros: P = 1 there, times dout = 0.
      const auto src = __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(stat_at), 0, rows_here * 4, 0x00020000);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (lds_void_ptr)(stat + (2 * stream + wave) * kWave), 4, lane * 4, 0, 0, 0);
    }
#endif
    if (load_turn < last_turn) {
      ++load_turn;
      q_at += q_turn;
      do_at += do_turn;
      stat_at += kTurnRows;
    } else {
      load_turn = 0;
      head += HEADS;
      start_head();
    }
  };
  auto load = [&](int i, uint8_t* qt, uint8_t* dot) __attribute__((always_inline)) {
#if defined(__HIP_DEVICE_COMPILE__)
    if (i < kLoads / 2)
      q_load.issue(q_src, i, rows_here, qt + stream * T::kBytes);
    else
      do_load.issue(do_src, i - kLoads / 2, rows_here, dot + stream * T::kBytes);
#endif
  };
  auto issue = [&](uint8_t* qt, uint8_t* dot, float* stat) __attribute__((always_inline)) {
    begin(stat);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) load(i, qt, dot);
  };
  // Scores and dout . v of a turn's rows.
  auto scores = [&](const uint8_t* qt, const uint8_t* dot, f32_x16& s, f32_x16& dp) __attribute__((always_inline)) {
#pragma unroll
    for (int r = 0; r < 16; ++r) s[r] = dp[r] = 0.0f;
#pragma unroll
    for (int kk = 0; kk < kDepth; ++kk) {
      multiply<BF16>(s, by_row.load(qt, 0, kk), k[kk]);
      multiply<BF16>(dp, by_row.load(dot, 0, kk), v[kk]);
    }
  };
  // The first turns of a head, whose rows do not all see the wave's last key;
  // of a head's rows from first_row on, those before see0 (+ 4 half) do not see the lane's.
  const int masked_turns = a.causal ? static_cast<int>(cut((wave_key + 31 - ahead - first_row + kTurnRows - 1) / kTurnRows, 0, per_head)) : 0;
  const int see0 = static_cast<int>(cut(key - ahead - first_row, 0, (wave + 2) * kTurnRows)) - 4 * half;
  // From a turn's scores to its probabilities (s) and dS (dp), then the sums;
  // the next turn's scores meanwhile, in one stretch of code without branches.
  auto step = [&](int i, const uint8_t* qt, const uint8_t* dot, const float* stat, const uint8_t* next_q, const uint8_t* next_do,
                  uint8_t* free_q, uint8_t* free_do, f32_x16& s, f32_x16& dp, f32_x16& next_s, f32_x16& next_dp) __attribute__((always_inline)) {
    float l[16], d[16];
    stat += stream * 2 * kWave;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const float4 ls = *reinterpret_cast<const float4*>(stat + 8 * g + 4 * half);
      const float4 dd = *reinterpret_cast<const float4*>(stat + kWave + 8 * g + 4 * half);
      l[4 * g] = ls.x, l[4 * g + 1] = ls.y, l[4 * g + 2] = ls.z, l[4 * g + 3] = ls.w;
      d[4 * g] = dd.x, d[4 * g + 1] = dd.y, d[4 * g + 2] = dd.z, d[4 * g + 3] = dd.w;
    }
    if (i < masked_turns) {
      const int see = see0 - i * kTurnRows;  // rows from here on see the key
#pragma unroll
      for (int r = 0; r < 16; ++r) l[r] = result_row(r) < see ? INFINITY : l[r];  // P = 0
    }
    constexpr int kColumns = BF16 ? 2 : 1;  // pairs of columns read ahead
    Operand<BF16> do_col[2 * kDt], q_col[2 * kDt];
    auto columns = [&](int n) __attribute__((always_inline)) {
      do_col[n] = by_column.load(dot, n / kDt, n % kDt);
      q_col[n] = by_column.load(qt, n / kDt, n % kDt);
    };
#pragma unroll
    for (int n = 0; n < kColumns; ++n) columns(n);
    if constexpr (BF16) pin();
    // A product of the next turn's scores, an operand's read two products
    // ahead, and a share of this turn's probabilities, in this order: the
    // matrix cores work on one product while the rest is issued.
    constexpr int kProducts = 2 * kDepth, kShare = 16 / kProducts ? 16 / kProducts : 1, kAhead = 3;
    auto operand = [&](int n) __attribute__((always_inline)) { return by_row.load(n & 1 ? next_do : next_q, 0, n >> 1); };
    Operand<BF16> ops[kProducts];
#pragma unroll
    for (int n = 0; n < kAhead; ++n) ops[n] = operand(n);
#pragma unroll
    for (int r = 0; r < 16; ++r) next_s[r] = next_dp[r] = 0.0f;
#pragma unroll
    for (int n = 0; n < kProducts; ++n) {
      static_assert(kProducts % kLoads == 0, "loads at even distances");
      if (n % (kProducts / kLoads) == 0) load(n / (kProducts / kLoads), free_q, free_do);
      if (n + kAhead < kProducts) ops[n + kAhead] = operand(n + kAhead);
      if (n & 1)
        multiply<BF16>(next_dp, ops[n], v[n >> 1]);
      else
        multiply<BF16>(next_s, ops[n], k[n >> 1]);
#pragma unroll
      for (int r = n * kShare; r < n * kShare + kShare; ++r) {
        s[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r], factor, -l[r]));
        if (r) dp[r - 1] = s[r - 1] * (dp[r - 1] - d[r - 1]);
      }
      if constexpr (BF16) pin();
    }
    dp[15] = s[15] * (dp[15] - d[15]);
    Operand<BF16> p[2], ds[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      p[h] = result_operand<BF16>(s, h);
      ds[h] = result_operand<BF16>(dp, h);
    }
#pragma unroll
    for (int n = 0; n < 2 * kDt; ++n) {
      const int h = n / kDt, dt = n % kDt;
      if (n + kColumns < 2 * kDt) columns(n + kColumns);
      multiply<BF16>(dv[dt], do_col[n], p[h]);
      multiply<BF16>(dk[dt], q_col[n], ds[h]);
      if constexpr (BF16) pin();
    }
  };
  int this_turn = 0;  // of its head
  // The turn in `qt`; the following one's rows are in next_q, and free_q, the turn before's, takes the one three ahead.
  auto turn = [&](const uint8_t* qt, const uint8_t* dot, const float* stat, const uint8_t* next_q, const uint8_t* next_do, uint8_t* free_q,
                  uint8_t* free_do, float* free_stat, f32_x16& s, f32_x16& dp, f32_x16& next_s, f32_x16& next_dp)
                  __attribute__((always_inline)) {
    // All but the youngest turn's loads: waves 0 and 1 have one more.
    if (wave < 2)
      wait_loads<kLoads + 1>();
    else
      wait_loads<kLoads>();
    __syncthreads();
    begin(free_stat);
    const int i = this_turn;
    this_turn = i == last_turn ? 0 : i + 1;
    step(i, qt, dot, stat, next_q, next_do, free_q, free_do, s, dp, next_s, next_dp);
  };

  // Turns by the ring's length, so that each place in it is an array of its own.
  if (turns > 0) {
    f32_x16 s_a, dp_a, s_b, dp_b;
    issue(q0, do0, stat0);
    issue(q1, do1, stat1);
    issue(q2, do2, stat2);
    wait_loads<0>();
    __syncthreads();
    scores(q0, do0, s_a, dp_a);
    for (int64_t u = 0; u < turns; u += 4) {
      turn(q0, do0, stat0, q1, do1, q3, do3, stat3, s_a, dp_a, s_b, dp_b);
      turn(q1, do1, stat1, q2, do2, q0, do0, stat0, s_b, dp_b, s_a, dp_a);
      turn(q2, do2, stat2, q3, do3, q1, do1, stat1, s_a, dp_a, s_b, dp_b);
      turn(q3, do3, stat3, q0, do0, q2, do2, stat2, s_b, dp_b, s_a, dp_a);
    }
    wait_loads<0>();  // none is under way into memory that is given back
  }
  if constexpr (HEADS == 2) {
    // The second stream's sums, 32 values of a head at a time, through shared memory.
    static_assert(kKeyWaves * kWave * 64 <= kBytes, "a part of dk fits a place of the ring");
    const int at = wave * kWave * 4 + lane;  // in 16 bytes, as 4 x 64 lanes
#pragma unroll
    for (int dt = 0; dt < kDt; ++dt) {
      __syncthreads();
      if (stream) {
        uint4 w[8];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          w[2 * g] = pack_piece<false>(reinterpret_cast<const float*>(&dk[dt]) + 4 * g);
          w[2 * g + 1] = pack_piece<false>(reinterpret_cast<const float*>(&dv[dt]) + 4 * g);
          reinterpret_cast<uint4*>(q0)[at + g * kWave] = w[2 * g];
          reinterpret_cast<uint4*>(do0)[at + g * kWave] = w[2 * g + 1];
        }
        hold_until_lds_written(w);
      }
      __syncthreads();
      if (!stream) {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          float x[4], y[4];
          unpack_piece<false>(reinterpret_cast<const uint4*>(q0)[at + g * kWave], x);
          unpack_piece<false>(reinterpret_cast<const uint4*>(do0)[at + g * kWave], y);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            dk[dt][4 * g + j] += x[j];
            dv[dt][4 * g + j] += y[j];
          }
        }
      }
    }
    if (stream) return;
  }
  store_columns<BF16, DP>(dk, a.scale, exists ? row_data(a.dk, seq.k0 + key, kv_head, kElem) : nullptr, a.head_dim, half);
  store_columns<BF16, DP>(dv, 1.0f, exists ? row_data(a.dv, seq.k0 + key, kv_head, kElem) : nullptr, a.head_dim, half);
}

int64_t k_tiles(const AttnSeqs& s, int per_tile) {
  return tile_bound(s, s.k_starts ? -1 : s.rows_k / s.n_seq, s.rows_k, per_tile);
}

// Two streams where a group has several heads and their rings fit shared memory.
bool two_streams(int group, int head_dim, bool bf16) { return group > 1 && (bf16 || head_dim <= 64); }

template <bool BF16, int DP>
hipError_t launch_at(const AttnArgs& a, hipStream_t stream) {
  const int group = a.q_heads / a.kv_heads;
  const int64_t tiles = q_tiles(a.seqs, group, kBlockRows);
  if (tiles)
    attention_dq_kernel<BF16, DP><<<dim3(static_cast<uint32_t>(tiles * a.kv_heads)), dim3(kWaves * kWave), 0, stream>>>(a);
  const bool two = two_streams(group, a.head_dim, BF16);
  const dim3 grid(static_cast<uint32_t>(k_tiles(a.seqs, (two ? 2 : 4) * kRows) * a.kv_heads)), block(kWaves * kWave);
  if (grid.x == 0) return hipGetLastError();
  if constexpr (BF16 || DP <= 64) {
    if (two) {
      attention_dkv_kernel<BF16, DP, 2><<<grid, block, 0, stream>>>(a);
      return hipGetLastError();
    }
  }
  attention_dkv_kernel<BF16, DP, 1><<<grid, block, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

int64_t attention_grad_workspace(const AttnSeqs& s, int q_heads, int kv_heads, int head_dim, bool bf16) {
  return 2 * s.rows_q * q_heads * 4;
}

int64_t attention_grad_blocks(const AttnSeqs& s, int q_heads, int kv_heads, int head_dim, bool bf16) {
  const int64_t q = q_tiles(s, q_heads / kv_heads, kBlockRows), k = k_tiles(s, 2 * kRows);
  return (q > k ? q : k) * kv_heads;
}

hipError_t launch_attention_grad(const AttnArgs& a, bool bf16, hipStream_t s) {
  if (bf16) return a.head_dim <= 64 ? launch_at<true, 64>(a, s) : launch_at<true, 128>(a, s);
  return a.head_dim <= 64 ? launch_at<false, 64>(a, s) : launch_at<false, 128>(a, s);
}

}  // namespace cq
