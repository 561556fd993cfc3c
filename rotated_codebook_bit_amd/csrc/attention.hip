// Attention over packed sequences, causal or not, with grouped heads, for
// prompts and for tokens that read a cache.
//
// For query i of a sequence and a query head of the group of key head h:
//   x_j = scale q . k_j,  p_j = exp(x_j - lse),  lse = log sum_j exp(x_j),  out = sum_j p_j v_j
// over the keys j it sees.  One pass over the keys: the running maximum and
// sum of each row stay in the lane that owns the row.
//
// Rows of a block are the queries of a whole group, (query, head) pairs with
// the head running fastest, so that a group's heads share each tile of keys.
// Scores are formed transposed, k . q^T, on the 32x32 matrix instructions: a
// lane then holds 16 scores of one row, the row's statistics need one
// exchange between the two halves of a wave, and the probabilities already
// lie as the second product's operand (out^T = v^T . p^T), which reads v by
// columns (attention.h).  Probabilities are rounded to bf16 for bf16 inputs
// (their sum is taken in float32 before): an error of half a step of each
// probability, as large as that of the stored output itself.
#include <algorithm>
#include <type_traits>

#include "attention.h"

namespace cq {
namespace {

// A row's running state, in powers of two: scores times scale * log2(e).
struct RowState {
  float top;  // the reference that probabilities are taken against
  float sum;  // of this lane's half of the keys
};

// Probabilities of SUBS x 32 scores against the running reference, which moves
// up (and the output with it) only when a row's maximum passes it by 2^8:
// below that the sums stay far from float32's limits, and the output's
// rescaling is left out for most tiles.
template <int SUBS, int DT>
__device__ __forceinline__ void soften(f32_x16 (&s)[SUBS], float factor, RowState& st, f32_x16 (&o)[DT]) {
  float top = s[0][0];
#pragma unroll
  for (int sub = 0; sub < SUBS; ++sub)
#pragma unroll
    for (int r = 0; r < 16; ++r) top = fmaxf(top, s[sub][r]);
  float a, b;
  both_halves(top, &a, &b);
  top = fmaxf(a, b) * factor;
  if (__any(top > st.top + 8.0f)) {
    const float up = fmaxf(top, st.top);
    const float shrink = st.top == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(st.top - up);
    st.sum *= shrink;
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
      for (int r = 0; r < 16; ++r) o[dt][r] *= shrink;
    st.top = up;
  }
  const float ref = st.top == -INFINITY ? 0.0f : st.top;  // no key seen yet: every score is -inf
#pragma unroll
  for (int sub = 0; sub < SUBS; ++sub)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[sub][r], factor, -ref));
      s[sub][r] = p;
      st.sum += p;
    }
}

constexpr int kWaves = 4;        // of a block
constexpr int kBlockRows = kWaves * kRows;
constexpr int kTileKeys = 64;

// Prompts: a block of 4 waves owns 128 rows and walks over tiles of 64 keys,
// the next tile on its way into the other half of shared memory meanwhile.
// Two blocks share a CU, so that one's exponentials run beside the other's
// products.  One prompt of 8192 tokens, 32 heads of 128 over 8, bf16: 520 to
// 543 us, 1.01 to 1.06 PFLOP/s, where a large library product reaches 1.36: the matrix cores are
// busy 60% of the cycles, the vector units 56%, shared memory's reads 30%, at the
// 2.1 GHz that the card holds under this load; a step that took a tenth of
// shared memory's cycles away left the time as it was and the clock lower.
template <bool BF16, int DP>
__global__ void __launch_bounds__(kWaves * kWave, BF16 ? 2 : 1) attention_kernel(AttnArgs a) {
  typedef Tile<BF16, DP, kTileKeys> T;
  constexpr int kElem = T::kElem, kSubs = kTileKeys / 32, kDepth = DP / 16, kDt = DP / 32;
  __shared__ __attribute__((aligned(16))) uint8_t k_tile0[T::kBytes], k_tile1[T::kBytes], v_tile0[T::kBytes], v_tile1[T::kBytes];
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), half = lane >> 5;
  const int group = a.q_heads / a.kv_heads;
  // Blocks in turn take the key heads, so that one head's keys stay in few
  // XCDs' caches, and the last rows of a sequence, which see most, come first.
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
  const int64_t all_see = r0 < rows ? keys_seen(seq, row_of(r0, rows, group).query, a.causal) : 0;  // keys that every row sees
  const int64_t seen = row.exists ? keys_seen(seq, row.query, a.causal) : 0;

  const uint8_t* const q_row =
      row.exists ? row_data(a.q, seq.q0 + row.query, static_cast<int64_t>(kv_head) * group + row.head, kElem) : nullptr;
  Operand<BF16> q[kDepth];
  load_row_operands<BF16, DP>(q_row, a.head_dim, half, q);

  const TileLoader<BF16, DP, kTileKeys, kWaves> k_load(wave, lane, a.k.row, a.head_dim), v_load(wave, lane, a.v.row, a.head_dim);
  const RowOperand<BF16, DP> by_row(lane);
  const ColumnOperand<BF16, DP> by_column(lane);
  [[maybe_unused]] const uint8_t* const k0 = row_data(a.k, seq.k0, kv_head, kElem);
  [[maybe_unused]] const uint8_t* const v0 = row_data(a.v, seq.k0, kv_head, kElem);
  const float factor = a.scale * kLog2e;

  RowState st{-INFINITY, 0.0f};
  f32_x16 o[kDt];
#pragma unroll
  for (int dt = 0; dt < kDt; ++dt)
#pragma unroll
    for (int r = 0; r < 16; ++r) o[dt][r] = 0.0f;

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
    f32_x16 s[kSubs];
#pragma unroll
    for (int sub = 0; sub < kSubs; ++sub)
#pragma unroll
      for (int r = 0; r < 16; ++r) s[sub][r] = 0.0f;
    constexpr int kAhead = 4;  // operands read before their product
    Operand<BF16> keys[kSubs * kDepth];
#pragma unroll
    for (int n = 0; n < kAhead; ++n) keys[n] = by_row.load(kt, n % kSubs, n / kSubs);
#pragma unroll
    for (int n = 0; n < kSubs * kDepth; ++n) {
      static_assert(kSubs * kDepth % kLoads == 0, "loads at even distances");
      if (n % (kSubs * kDepth / kLoads) == 0) load(n / (kSubs * kDepth / kLoads), next_k, next_v);
      if (n + kAhead < kSubs * kDepth) keys[n + kAhead] = by_row.load(kt, (n + kAhead) % kSubs, (n + kAhead) / kSubs);
      multiply<BF16>(s[n % kSubs], keys[n], q[n / kSubs]);
      if constexpr (BF16) pin();
    }
    if (key + kTileKeys > all_see) {
      const int left = static_cast<int>(min(seen - key, int64_t(kTileKeys))) - 4 * half;
#pragma unroll
      for (int sub = 0; sub < kSubs; ++sub)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (32 * sub + result_row(r) >= left) s[sub][r] = -INFINITY;
    }
    soften<kSubs, kDt>(s, factor, st, o);
    Operand<BF16> values[2 * kSubs * kDt];
#pragma unroll
    for (int n = 0; n < kDt; ++n) values[n] = by_column.load(vt, n / kDt, n % kDt);
#pragma unroll
    for (int step = 0; step < 2 * kSubs; ++step) {
      const Operand<BF16> p = result_operand<BF16>(s[step / 2], step % 2);
#pragma unroll
      for (int dt = 0; dt < kDt; ++dt) {
        const int n = step * kDt + dt;
        if (step + 1 < 2 * kSubs) values[n + kDt] = by_column.load(vt, step + 1, dt);
        multiply<BF16>(o[dt], values[n], p);
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

  float sum_a, sum_b;
  both_halves(st.sum, &sum_a, &sum_b);
  const float sum = sum_a + sum_b;
  const int64_t out_row = seq.q0 + row.query, out_head = static_cast<int64_t>(kv_head) * group + row.head;
  store_columns<BF16, DP>(o, sum == 0.0f ? 0.0f : 1.0f / sum, row.exists ? row_data(a.out, out_row, out_head, kElem) : nullptr,
                          a.head_dim, half);
  if (a.lse && row.exists && half == 0)
    a.lse[out_row * a.q_heads + out_head] = sum == 0.0f ? -INFINITY : (st.top + __builtin_log2f(sum)) * kLn2;
}

// ---- Few rows: the keys split over waves and blocks -------------------------------

constexpr int kPieceKeys = 2048;

// Keys of a split of a tile of rows whose last row sees `keys`: the usual
// number of pieces, or as many as the grid has of half of kPieceKeys.
__device__ __forceinline__ int64_t split_keys(int64_t keys, const AttnArgs& a, int step) {
  const uint32_t n = static_cast<uint32_t>(keys), half = kPieceKeys / 2;
  const uint32_t pieces = min(max(static_cast<uint32_t>(a.pieces), (n + half - 1) / half), static_cast<uint32_t>(a.splits));
  const uint32_t each = (n + pieces - 1) / pieces;
  return static_cast<int64_t>((each + step - 1) / step * step);
}

template <bool BF16, int DP>
struct SplitShape {
  // bf16: two tiles of keys and of values per wave, as memory bounds it.  Float32:
  // one of each, as it is bound by the matrix cores and needs a wave for each
  // SIMD.  Blocks are small enough that two share a CU, so that one's start and
  // end run beside the other's stream of keys.
  static constexpr int kTile = Tile<BF16, DP, 32>::kBytes, kBuffers = BF16 ? 2 : 1;
  static constexpr int kWaves = !BF16 && DP == 64 ? 4 : 2;
  static constexpr int kStep = 32 * kWaves;  // keys that a block takes in one turn
  static constexpr int kPitch = DP + 4;      // floats per row of a wave's output in shared memory
  static constexpr int kPart = kRows * kPitch * 4;
  // Each of two arrays: keys and values of a turn of all waves (bf16), or all keys or all values (float32).
  static constexpr int kArray = kWaves * kBuffers * kTile;
  static_assert(kWaves / 2 * kPart <= kArray, "half of the waves' outputs fit one of the arrays");
};

// A block takes one tile of up to 32 rows and one split of its keys; each wave
// walks over its own tiles of 32 keys, which only it loads and reads, so no
// wave waits for another before the end.  64 tokens over caches of up to 8192 keys
// (1.3 GB, bf16): 256 us, 5.1 TB/s, a large copy's rate; one token over 8192 keys:
// 12.4 us for 34 MB, start and end of 512 blocks.  Float32, heads of 128, 2.0 GB:
// 424 us, 4.7 TB/s (806 with two tiles of each per wave and half the waves).
template <bool BF16, int DP>
__global__ void __launch_bounds__((SplitShape<BF16, DP>::kWaves * kWave), (SplitShape<BF16, DP>::kWaves / 2)) attention_split_kernel(AttnArgs a) {
  typedef SplitShape<BF16, DP> Shape;
  typedef Tile<BF16, DP, 32> T;
  constexpr int kElem = T::kElem, kDepth = DP / 16, kDt = DP / 32, W = Shape::kWaves;
  // Two arrays, not one indexed by the turn: the compiler has to see that the
  // loads under way do not meet the tile being read, or waits for them.
  __shared__ __attribute__((aligned(16))) uint8_t tiles0[Shape::kArray], tiles1[Shape::kArray];
  __shared__ float tops[W][kRows], sums[W][kRows];
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), half = lane >> 5;
  const int group = a.q_heads / a.kv_heads;
  // Pieces that a tile may not have come behind those that all have: among them
  // they would leave the last of those few places of the card at a time.
  const uint32_t units = gridDim.x / a.splits, sure = units * a.pieces, at = blockIdx.x;
  const uint32_t unit = at < sure ? at / a.pieces : (at - sure) % units;
  const int split = static_cast<int>(at < sure ? at % a.pieces : a.pieces + (at - sure) / units);
  const int kv_head = static_cast<int>(unit % a.kv_heads);
  SeqRows seq;
  int64_t tile;
  if (!find_tile<true, !BF16>(a.seqs, unit / a.kv_heads,
                 [&](const SeqRows& s) { return (s.nq * group + kRows - 1) / kRows; }, &seq, &tile))
    return;
  const int64_t rows = seq.nq * group, r0 = tile * kRows;
  const int64_t keys = keys_seen(seq, row_of(min(r0 + kRows, rows) - 1, rows, group).query, a.causal);
  const int64_t each = split_keys(keys, a, Shape::kStep);
  const int64_t begin = split * each, end = min(begin + each, keys);
  if (split > 0 && begin >= keys) return;  // the first split writes rows that see nothing
  const Row row = row_of(r0 + (lane & 31), rows, group);
  const int64_t all_see = keys_seen(seq, row_of(r0, rows, group).query, a.causal);
  const int64_t seen = row.exists ? keys_seen(seq, row.query, a.causal) : 0;
  const int64_t out_row = seq.q0 + row.query, out_head = static_cast<int64_t>(kv_head) * group + row.head;

  const TileLoader<BF16, DP, 32, 1> k_load(0, lane, a.k.row, a.head_dim), v_load(0, lane, a.v.row, a.head_dim);
  constexpr int kLoads = TileLoader<BF16, DP, 32, 1>::kLoads;  // of a tile
  const RowOperand<BF16, DP> by_row(lane);
  const ColumnOperand<BF16, DP> by_column(lane);
  const uint8_t* const k0 = row_data(a.k, seq.k0, kv_head, kElem);
  const uint8_t* const v0 = row_data(a.v, seq.k0, kv_head, kElem);
  const float factor = a.scale * kLog2e;

  uint8_t* const even = tiles0 + wave * Shape::kBuffers * T::kBytes;
  uint8_t* const odd = tiles1 + wave * Shape::kBuffers * T::kBytes;
  auto load_k = [&](int64_t key, uint8_t* kt) __attribute__((always_inline)) {
    k_load.issue(k0 + key * a.k.row * kElem, key < end ? seq.nk - key : 0, kt);
  };
  auto load_v = [&](int64_t key, uint8_t* vt) __attribute__((always_inline)) {
    v_load.issue(v0 + key * a.v.row * kElem, key < end ? seq.nk - key : 0, vt);
  };
  int64_t key = begin + 32 * wave;
  load_k(key, even);
  load_v(key, BF16 ? even + T::kBytes : odd);
  Operand<BF16> q[kDepth];
  load_row_operands<BF16, DP>(row.exists ? row_data(a.q, out_row, out_head, kElem) : nullptr, a.head_dim, half, q);
  RowState st{-INFINITY, 0.0f};
  f32_x16 o[kDt];
#pragma unroll
  for (int dt = 0; dt < kDt; ++dt)
#pragma unroll
    for (int r = 0; r < 16; ++r) o[dt][r] = 0.0f;
  auto scores = [&](int64_t key, const uint8_t* kt, f32_x16 (&s)[1]) __attribute__((always_inline)) {
#pragma unroll
    for (int r = 0; r < 16; ++r) s[0][r] = 0.0f;
#pragma unroll
    for (int kk = 0; kk < kDepth; ++kk) multiply<BF16>(s[0], by_row.load(kt, 0, kk), q[kk]);
    if (key + 32 > min(all_see, end)) {
      const int left = static_cast<int>(min(min(seen, end) - key, int64_t(32))) - 4 * half;
#pragma unroll
      for (int r = 0; r < 16; ++r)
        if (result_row(r) >= left) s[0][r] = -INFINITY;
    }
  };
  auto add_values = [&](const f32_x16 (&s)[1], const uint8_t* vt) __attribute__((always_inline)) {
#pragma unroll
    for (int step = 0; step < 2; ++step) {
      const Operand<BF16> p = result_operand<BF16>(s[0], step);
      Operand<BF16> rest;
      if constexpr (BF16) {
        // What the rounding left: memory bounds this kernel, the second product is free.
        f32_x16 left;
#pragma unroll
        for (int j = 0; j < 8; ++j) left[8 * step + j] = s[0][8 * step + j] - static_cast<float>(p[j]);
        rest = result_operand<BF16>(left, step);
      }
#pragma unroll
      for (int dt = 0; dt < kDt; ++dt) {
        const Operand<BF16> v = by_column.load(vt, step, dt);
        multiply<BF16>(o[dt], v, p);
        if constexpr (BF16) multiply<BF16>(o[dt], v, rest);
      }
    }
  };

  if constexpr (BF16) {
    // One turn's loads are under way while the turn before is computed.
    auto turn = [&](int64_t key, const uint8_t* now, uint8_t* next) __attribute__((always_inline)) {
      if (key + Shape::kStep < end) {
        wait_lds_writes();  // the last turn's reads of the other half are done
        load_k(key + Shape::kStep, next);
        load_v(key + Shape::kStep, next + T::kBytes);
        wait_loads<2 * kLoads>();
      } else {
        wait_loads<0>();
      }
      f32_x16 s[1];
      scores(key, now, s);
      soften<1, kDt>(s, factor, st, o);
      add_values(s, now + T::kBytes);
    };
    while (key < end) {
      turn(key, even, odd);
      key += Shape::kStep;
      if (key >= end) break;
      turn(key, odd, even);
      key += Shape::kStep;
    }
  } else {
    // The next keys are under way once these scores are formed, the next values
    // once these are added.  Past the end: zeros, which nothing reads.
    for (; key < end; key += Shape::kStep) {
      f32_x16 s[1];
      wait_loads<kLoads>();  // all but the values
      scores(key, even, s);
      wait_lds_writes();  // every read of the keys is done
      load_k(key + Shape::kStep, even);
      soften<1, kDt>(s, factor, st, o);
      wait_loads<kLoads>();  // all but the next keys
      add_values(s, odd);
      wait_lds_writes();
      load_v(key + Shape::kStep, odd);
    }
  }
  wait_loads<0>();  // none is under way into memory that is used again

  // The waves' rows together: each leaves its output, maximum and sum.
  auto part_of = [&](int w) __attribute__((always_inline)) {
    return reinterpret_cast<float*>((w % 2 ? tiles1 : tiles0) + w / 2 * Shape::kPart);
  };
  float* const part = part_of(wave);
  float sum_a, sum_b;
  both_halves(st.sum, &sum_a, &sum_b);
  const float sum = sum_a + sum_b;
  __syncthreads();  // every wave has read its tiles
#pragma unroll
  for (int dt = 0; dt < kDt; ++dt) {
    uint4 w[4];
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      w[g] = pack_piece<false>(reinterpret_cast<const float*>(&o[dt]) + 4 * g);
      *reinterpret_cast<uint4*>(part + (lane & 31) * Shape::kPitch + 32 * dt + 8 * g + 4 * half) = w[g];
    }
    hold_until_lds_written(w);
  }
  if (half == 0) {
    tops[wave][lane] = st.top;
    sums[wave][lane] = sum;
    wait_lds_writes();
    hold_value(st.top);
    hold_value(sum);
  }
  __syncthreads();
  constexpr int kQuads = DP / 4;
  for (int i = threadIdx.x; i < kRows * kQuads; i += W * kWave) {
    const int r = i / kQuads, d = i % kQuads * 4;
    const Row w = row_of(r0 + r, rows, group);
    if (!w.exists || d >= a.head_dim) continue;
    float top = tops[0][r];
#pragma unroll
    for (int j = 1; j < W; ++j) top = fmaxf(top, tops[j][r]);
    float total = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < W; ++j) {
      const float share = tops[j][r] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(tops[j][r] - top);
      total = __builtin_fmaf(share, sums[j][r], total);
      const float4 v = *reinterpret_cast<const float4*>(part_of(j) + r * Shape::kPitch + d);
      acc[0] = __builtin_fmaf(share, v.x, acc[0]);
      acc[1] = __builtin_fmaf(share, v.y, acc[1]);
      acc[2] = __builtin_fmaf(share, v.z, acc[2]);
      acc[3] = __builtin_fmaf(share, v.w, acc[3]);
    }
    const int64_t at = (seq.q0 + w.query) * a.q_heads + static_cast<int64_t>(kv_head) * group + w.head;
    if (a.splits > 1) {
      // A sequence of rows: [split][row and head][head_dim + 4], output, maximum, sum.
      float* const p = a.ws + (split * a.seqs.rows_q * a.q_heads + at) * (a.head_dim + 4);
      *reinterpret_cast<float4*>(p + d) = make_float4(acc[0], acc[1], acc[2], acc[3]);
      if (d == 0) *reinterpret_cast<float2*>(p + a.head_dim) = make_float2(top, total);
    } else {
      const float inv = total == 0.0f ? 0.0f : 1.0f / total;
      uint8_t* const out = row_data(a.out, seq.q0 + w.query, static_cast<int64_t>(kv_head) * group + w.head, kElem) + d * kElem;
      if constexpr (BF16)
        *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv));
      else
        *reinterpret_cast<float4*>(out) = make_float4(acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv);
      if (a.lse && d == 0) a.lse[at] = total == 0.0f ? -INFINITY : (top + __builtin_log2f(total)) * kLn2;
    }
  }
}

// Joins the splits' shares of the rows of a tile: a wave takes a row, lane s
// the maximum and sum of split s, then teams of lanes of 4 values every
// (64 / team)-th split each.  Latency: 6 to 8 us for 64 rows of 4 splits or one
// row of 64 (16 or 32 loads ahead instead of 8: 7.4, 9.1).
template <bool BF16, int DP>
__global__ void __launch_bounds__(256) attention_join_kernel(AttnArgs a) {
  constexpr int kElem = BF16 ? 2 : 4, kQuads = DP / 4, kTeams = kWave / kQuads;
  const int lane = threadIdx.x & (kWave - 1), team = lane / kQuads;
  const int group = a.q_heads / a.kv_heads;
  const int kv_head = static_cast<int>(blockIdx.x % a.kv_heads);
  SeqRows seq;
  int64_t tile;
  if (!find_tile<true, false>(a.seqs, blockIdx.x / a.kv_heads, [&](const SeqRows& s) { return (s.nq * group + kRows - 1) / kRows; }, &seq, &tile))
    return;
  const int64_t rows = seq.nq * group, r0 = tile * kRows;
  const int64_t keys = keys_seen(seq, row_of(min(r0 + kRows, rows) - 1, rows, group).query, a.causal);
  const int64_t each = split_keys(keys, a, SplitShape<BF16, DP>::kStep);
  const int live = keys <= each ? 1 : static_cast<int>((keys + each - 1) / each);
  const int d = lane % kQuads * 4;
  const int64_t pitch = a.head_dim + 4, step = a.seqs.rows_q * a.q_heads * pitch;
  for (int r = threadIdx.x / kWave; r < kRows && r0 + r < rows; r += 256 / kWave) {
    const Row w = row_of(r0 + r, rows, group);
    const int64_t head = static_cast<int64_t>(kv_head) * group + w.head, at = (seq.q0 + w.query) * a.q_heads + head;
    const float* const p = a.ws + at * pitch;
    float top = -INFINITY, sum = 0.0f;
    if (lane < live) {
      const float2 ms = *reinterpret_cast<const float2*>(p + lane * step + a.head_dim);
      top = ms.x;
      sum = ms.y;
    }
    float best = top;
#pragma unroll
    for (int x = 1; x < kWave; x <<= 1) best = fmaxf(best, __shfl_xor(best, x));
    const float share = top == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(top - best);
    const float total = wave_sum(share * sum);
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    const bool inside = d < a.head_dim;
    constexpr int kAhead = 8;  // loads in flight
    for (int s = team; s < live + team; s += kAhead * kTeams) {
      float4 v[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int split = s + i * kTeams;
        v[i] = inside && split < live ? *reinterpret_cast<const float4*>(p + split * step + d) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int split = s + i * kTeams;
        const float f = __shfl(share, split < live ? split : kWave - 1);
        if (split >= live) continue;
        acc[0] = __builtin_fmaf(f, v[i].x, acc[0]);
        acc[1] = __builtin_fmaf(f, v[i].y, acc[1]);
        acc[2] = __builtin_fmaf(f, v[i].z, acc[2]);
        acc[3] = __builtin_fmaf(f, v[i].w, acc[3]);
      }
    }
#pragma unroll
    for (int x = kQuads; x < kWave; x <<= 1)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] += __shfl_xor(acc[j], x);
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    if (inside && team == 0) {
      uint8_t* const out = row_data(a.out, seq.q0 + w.query, head, kElem) + d * kElem;
      if constexpr (BF16)
        *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv));
      else
        *reinterpret_cast<float4*>(out) = make_float4(acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv);
    }
    if (a.lse && lane == 0) a.lse[at] = total == 0.0f ? -INFINITY : (best + __builtin_log2f(total)) * kLn2;
  }
}

constexpr int kMostSplits = kWave;  // a lane of the joining wave each

// Float32 prompts in at most two 128-row blocks per CU: the matrix cores'
// float32 rate bounds them, so the block with the most keys, 69 ns each (heads of
// 64; 280 of 128), ends last.  The split kernel deals them to 4 waves (2) and four
// times the blocks, but takes some 8 us more.  Split (128-row blocks), 8 heads of 64
// over 2: one prompt of 4096 tokens 167 us (284), 3 of 8192 in all 249 (354), 13 of 4001
// 41 (66); 32 heads of 64 over 8, 16 of 8192 in all (more blocks): 324 (249).  Heads of
// 128: 6 of 3000 in all, 4 heads over 1, 67 (146); 16 of 64 rows over 4096 keys of 8
// heads 191 (557); one of 4096, 32 heads over 8, 1333 (1185).
bool float_prompts(const AttnSeqs& s, int group, int kv_heads, bool bf16) {
  return !bf16 && s.rows_q * group > kRows * s.n_seq && s.rows_k >= 256 * s.n_seq && s.rows_q * group * kv_heads <= 2 * kCus * kBlockRows;
}

// Whether a call takes the split kernel.  Up to 32 rows per sequence and key
// head (one tile) do: of every sequence, or (q_starts) on the average, unless one
// sequence may have most of many rows.  For that one 128-row blocks read its keys a
// quarter as often, and for the others they are no slower: bf16, 32 heads of 128 over 8,
// 128-row blocks (split kernel): a prompt of 8192 tokens and 300 of 1, over 4096 keys each,
// 1393 us (2160), of 1024 902 (1025), 512 x 5 tokens over 2048 823 (846); without caches,
// 32 heads over 32, 8192 tokens in 257 sequences 152 (270), one of 8192 and 300 of 1 674
// (1460).  Float32 is bound by the matrix cores, whose work the padded rows are: the
// same 10599 (6595), 5614 (1893), 4636 (1560), 597 (407), 5180 (4921).
// More rows do while 128-row blocks would leave most of the card idle over long keys:
// a block takes 18 ns per key (bf16 heads of 128, 512 blocks at once), a tile of 32 rows
// some 60 us per 2^20 keys of all CUs, and 20 us more to start, end and join.  Over
// 8192 keys of 8 heads, 32 query heads, split kernel (128-row blocks): 64 new tokens
// 49 us (136), 128 68 (135), 512 196 (138); 8 x 16 over 4096 49 (71); 1000 tokens of a
// prompt, 8 heads of 64 over 2, 30 (17).
constexpr int64_t kFewTiles = 4 * kCus;  // of 32 rows, all full
bool few_rows(const AttnSeqs& s, int group, int kv_heads, bool bf16) {
  const int64_t rows = s.rows_q * group;
  const bool may_be_one = bf16 && s.q_starts && s.rows_q > s.n_seq && rows * kv_heads > kFewTiles * kRows;
  if ((rows <= kRows * s.n_seq && !may_be_one) || float_prompts(s, group, kv_heads, bf16)) return true;
  const int64_t keys = s.rows_k / s.n_seq, blocks = q_tiles(s, group, kBlockRows) * kv_heads;
  const int64_t units = q_tiles(s, group, kRows) * kv_heads;
  return keys > 0 && units + 333000 / keys < 300 * ceil_div(blocks, 2 * kCus);
}

int split_step(int head_dim, bool bf16) {
  if (bf16) return head_dim <= 64 ? SplitShape<true, 64>::kStep : SplitShape<true, 128>::kStep;
  return head_dim <= 64 ? SplitShape<false, 64>::kStep : SplitShape<false, 128>::kStep;
}

template <bool BF16, int DP>
hipError_t launch_at(const AttnArgs& a, hipStream_t stream) {
  const int group = a.q_heads / a.kv_heads;
  if (!few_rows(a.seqs, group, a.kv_heads, BF16)) {
    const int64_t tiles = q_tiles(a.seqs, group, kBlockRows);
    attention_kernel<BF16, DP><<<dim3(static_cast<uint32_t>(tiles * a.kv_heads)), dim3(kWaves * kWave), 0, stream>>>(a);
    return hipGetLastError();
  }
  const int64_t units = q_tiles(a.seqs, group, kRows) * a.kv_heads;
  attention_split_kernel<BF16, DP>
      <<<dim3(static_cast<uint32_t>(units * a.splits)), dim3(SplitShape<BF16, DP>::kWaves * kWave), 0, stream>>>(a);
  if (a.splits > 1) attention_join_kernel<BF16, DP><<<dim3(static_cast<uint32_t>(units)), dim3(256), 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

// Splits of the keys: two blocks per CU where tiles of rows alone are fewer, and
// pieces of at most 2048 keys (64 pieces at most), so that sequences of different
// lengths do not leave the card to the longest (64 tokens over up to 8192 keys of 8 heads, bf16: 238
// us in pieces of 4096, 227 of 2048, 252 of 512).  More blocks than fit at once
// each pay their start again (16 tokens over 2048 keys: 512 blocks 31 us, 2048 46).
// Float32 prompts are not cut by length: their rows, not their keys, fill the card.
//
// That is for a sequence of the mean length, within 16 rounds of the card (a
// cache may be larger than what it holds).  With k_starts one sequence may have
// nearly all keys: a tile with more than the mean's is cut further by its own
// length (split_keys), as the grid has blocks for all keys in one sequence, within
// 4 rounds; those that a tile does not use have to start all the same.  bf16, 32
// heads of 128 over 8, by k_lens alone and by k_starts too: 64 tokens over up to 8192
// keys 232 and 232 us, 256 over up to 4096 427 and 430, 16 over 2048 32 and 37, 8 over 8192 53
// and 58; all of the same in 1, 2, 4, 8 and 16 pieces, 64 tokens over one cache of 8192 keys
// and 63 of 100: 159, 92, 55, 75, 121.
AttnSplits attention_splits(const AttnSeqs& s, int q_heads, int kv_heads, int head_dim, bool bf16) {
  const int group = q_heads / kv_heads;
  if (!few_rows(s, group, kv_heads, bf16)) return {1, 1};
  const int64_t units = q_tiles(s, group, kRows) * kv_heads, step = split_step(head_dim, bf16), fill = ceil_div(2 * kCus, units);
  const int64_t mean = ceil_div(s.rows_k, s.n_seq), longest = s.k_starts ? s.rows_k : mean;
  // As many as wanted, of at least two steps of `keys`.
  auto pieces = [&](int64_t wanted, int64_t keys) {
    return static_cast<int>(std::max(std::min({wanted, ceil_div(keys, 2 * step), int64_t(kMostSplits)}), int64_t(1)));
  };
  auto by_length = [&](int64_t keys, int64_t rounds) { return std::min(ceil_div(keys, kPieceKeys), (rounds * 2 * kCus + units / 2) / units); };
  if (float_prompts(s, group, kv_heads, bf16)) return {pieces(fill, longest), pieces(fill, longest)};
  const int usual = pieces(std::max(fill, by_length(mean, 16)), mean);
  return {usual, std::max(usual, pieces(by_length(longest, 4), longest))};
}

int64_t attention_workspace(const AttnSeqs& s, int q_heads, int kv_heads, int head_dim, bool bf16) {
  const int splits = attention_splits(s, q_heads, kv_heads, head_dim, bf16).splits;
  return splits > 1 ? splits * s.rows_q * q_heads * (head_dim + 4) * 4 : 0;
}

int64_t attention_blocks(const AttnSeqs& s, int q_heads, int kv_heads, int head_dim, bool bf16) {
  const int group = q_heads / kv_heads;
  if (!few_rows(s, group, kv_heads, bf16)) return q_tiles(s, group, kBlockRows) * kv_heads;
  return q_tiles(s, group, kRows) * kv_heads * attention_splits(s, q_heads, kv_heads, head_dim, bf16).splits;
}

hipError_t launch_attention(const AttnArgs& a, bool bf16, hipStream_t s) {
  if (bf16) return a.head_dim <= 64 ? launch_at<true, 64>(a, s) : launch_at<true, 128>(a, s);
  return a.head_dim <= 64 ? launch_at<false, 64>(a, s) : launch_at<false, 128>(a, s);
}

}  // namespace cq
