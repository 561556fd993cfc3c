// What the attention kernels share: the sequences of a packed batch, tiles of
// keys or queries in shared memory, and their operands for the matrix cores.
#pragma once

#include "lanes.h"

namespace cq {

typedef __bf16 bf16_x8 __attribute__((ext_vector_type(8)));
typedef float f32_x8 __attribute__((ext_vector_type(8)));
typedef float f32_x16 __attribute__((ext_vector_type(16)));
typedef short s16_x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void* lds_void_ptr;
typedef __attribute__((address_space(3))) s16_x4* lds_s16x4_ptr;

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// ---- Sequences -------------------------------------------------------------------

// Rows of one sequence.
struct SeqRows {
  int64_t q0, nq, k0, nk;
};

__device__ __forceinline__ int64_t seq_index(const void* p, int bytes, int64_t i) {
  return bytes == 4 ? static_cast<const int32_t*>(p)[i] : static_cast<const int64_t*>(p)[i];
}
__device__ __forceinline__ int64_t cut(int64_t v, int64_t lo, int64_t hi) { return v < lo ? lo : v > hi ? hi : v; }

// Offsets come from device memory, which the host cannot check: whatever they
// hold, the rows they give lie inside the tensors.
__device__ __forceinline__ SeqRows seq_rows(const AttnSeqs& a, int64_t s) {
  SeqRows r;
  if (a.q_starts) {
    r.q0 = cut(seq_index(a.q_starts, a.index_bytes, s), 0, a.rows_q);
    r.nq = cut(seq_index(a.q_starts, a.index_bytes, s + 1), r.q0, a.rows_q) - r.q0;
  } else {
    r.nq = a.rows_q / a.n_seq;
    r.q0 = s * r.nq;
  }
  if (a.k_starts) {
    r.k0 = cut(seq_index(a.k_starts, a.index_bytes, s), 0, a.rows_k);
    r.nk = a.k_lens ? cut(seq_index(a.k_lens, a.index_bytes, s), 0, a.rows_k - r.k0)
                    : cut(seq_index(a.k_starts, a.index_bytes, s + 1), r.k0, a.rows_k) - r.k0;
  } else {
    const int64_t each = a.rows_k / a.n_seq;
    r.k0 = s * each;
    r.nk = a.k_lens ? cut(seq_index(a.k_lens, a.index_bytes, s), 0, each) : each;
  }
  return r;
}

// A value that all lanes agree on, for the compiler to know it.
__device__ __forceinline__ int64_t uniform(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<int>(v));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<int>(v >> 32));
  return static_cast<int64_t>(static_cast<uint64_t>(hi) << 32 | lo);
}

// The t-th tile to run, if sequence s has count(seq_rows(s)) tiles; false past
// the last one.  LAST_FIRST: a tile's work grows with its number, as a row's keys do;
// otherwise with how many follow it, as a key's rows do.  Tiles with more to do
// come first: within a sequence, or (SORTED, up to 64 sequences) over all of them,
// so that no long block starts when the others end.  That takes 1 us per block
// and walks over all sequences' keys at once, which pays where a CU runs one block at
// a time (gradient of keys and values, float32: 8192 tokens in 16 sequences, 32 heads
// of 128 over 8, gradients 225 -> 209 us, float32 1639 -> 1238; but bf16 forward 64 -> 74)
// and where the matrix cores bound the blocks (float32 split kernel, 13 prompts of 4001
// tokens, 8 heads of 64 over 2, 49 -> 41; no change where memory does).
// More sequences are walked 64 at a time by every wave, some 0.5 us a turn: little
// up to some hundreds (512 sequences of 64 tokens, 32 heads of 128 over 8, bf16: 182 us
// of which 31), most of the time for thousands (4096 of 16: 1662, of which 1200).
// All lanes of a wave take part and agree on the result.
template <bool LAST_FIRST, bool SORTED, class Count>
__device__ __forceinline__ bool find_tile(const AttnSeqs& a, int64_t t, Count count, SeqRows* rows, int64_t* tile) {
  const int lane = threadIdx.x & (kWave - 1);
  if (a.n_seq == 1) {
    const SeqRows one = seq_rows(a, 0);
    *rows = SeqRows{uniform(one.q0), uniform(one.nq), uniform(one.k0), uniform(one.nk)};
    const int64_t tiles = uniform(count(*rows));
    *tile = LAST_FIRST ? tiles - 1 - t : t;
    return t < tiles;
  }
  auto take = [&](const SeqRows& mine, int at) __attribute__((always_inline)) {
    *rows = SeqRows{uniform(__shfl(mine.q0, at)), uniform(__shfl(mine.nq, at)), uniform(__shfl(mine.k0, at)),
                    uniform(__shfl(mine.nk, at))};
  };
  if (SORTED && a.n_seq <= kWave) {
    SeqRows mine{0, 0, 0, 0};
    int tiles = 0;
    if (lane < a.n_seq) {
      mine = seq_rows(a, lane);
      tiles = static_cast<int>(count(mine));
    }
    // Tiles of at least a rank, the work's place 1, 2, ... in the sequence.  A grid
    // has at most 2^24 blocks: float32 counts them exactly.
    auto from = [&](int rank) __attribute__((always_inline)) {
      return __builtin_amdgcn_readfirstlane(static_cast<int>(wave_sum(static_cast<float>(tiles >= rank ? tiles - rank + 1 : 0))));
    };
    if (t >= from(1)) return false;
    const int number = static_cast<int>(t);
    int low = 1, high = tiles;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) high = max(high, __shfl_xor(high, d));
    high = __builtin_amdgcn_readfirstlane(high);
    while (low < high) {  // the highest rank that more than t tiles reach
      const int middle = (low + high + 1) / 2;
      if (from(middle) > number)
        low = middle;
      else
        high = middle - 1;
    }
    const uint64_t there = __ballot(tiles >= low);
    const int before = __builtin_popcountll(there & ((uint64_t(1) << lane) - 1)), left = number - from(low + 1);
    const uint64_t it = __ballot(tiles >= low && before == left);
    if (!it) return false;  // starts that do not ascend: more tiles than are counted exactly
    const int at = __builtin_ctzll(it);
    *tile = LAST_FIRST ? low - 1 : __builtin_amdgcn_readfirstlane(__shfl(tiles, at)) - low;
    take(mine, at);
    return true;
  }
  for (int64_t base = 0; base < a.n_seq; base += kWave) {
    const int64_t s = base + lane;
    SeqRows mine{0, 0, 0, 0};
    if (s < a.n_seq) mine = seq_rows(a, s);
    const int64_t c = s < a.n_seq ? count(mine) : 0;
    int64_t upto = c;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const int64_t v = __shfl_up(upto, d);
      if (lane >= d) upto += v;
    }
    const int64_t total = uniform(__shfl(upto, kWave - 1));
    if (t < total) {
      const int at = __builtin_ctzll(__ballot(upto > t));
      *tile = LAST_FIRST ? uniform(__shfl(upto, at)) - 1 - t : t - uniform(__shfl(upto - c, at));
      take(mine, at);
      return true;
    }
    t -= total;
  }
  return false;
}

// Keys that query i of a sequence sees.
__device__ __forceinline__ int64_t keys_seen(const SeqRows& r, int64_t i, bool causal) {
  return causal ? cut(i + r.nk - r.nq + 1, 0, r.nk) : r.nk;
}

// ---- Rows of a group -------------------------------------------------------------

constexpr int kRows = 32;  // rows of a wave: the columns of a 32 x 32 result

// Row r of a group's rows: its query and head.
struct Row {
  int64_t query;
  int head;
  bool exists;
};
__device__ __forceinline__ Row row_of(int64_t r, int64_t rows, int group) {
  Row w;
  w.exists = r < rows;
  const uint64_t at = static_cast<uint64_t>(w.exists ? r : 0);
  w.query = at <= 0xFFFFFFFFu ? static_cast<uint32_t>(at) / static_cast<uint32_t>(group) : at / group;
  w.head = static_cast<int>(at - static_cast<uint64_t>(w.query) * group);
  return w;
}

__device__ __forceinline__ uint8_t* row_data(const HeadRows& t, int64_t row, int64_t head, int elem) {
  return t.data + (row * t.row + head * t.head) * elem;
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Bound on the tiles of `rows` rows per tile over all sequences.
inline int64_t tile_bound(const AttnSeqs& s, int64_t rows_each, int64_t rows, int64_t per_tile) {
  if (rows_each >= 0) return s.n_seq * ceil_div(rows_each, per_tile);
  return rows / per_tile + s.n_seq;
}
inline int64_t q_tiles(const AttnSeqs& s, int group, int per_tile) {
  return tile_bound(s, s.q_starts ? -1 : s.rows_q / s.n_seq * group, s.rows_q * group, per_tile);
}

// ---- Operands --------------------------------------------------------------------

// An operand of 32 rows by 16 values of the summed axis: lane l holds 8 values
// of row l % 32, half l / 32 of the 16.  Float32 takes eight products of depth
// 2 where bf16 takes one of depth 16, element j of both halves at a time, so
// both types share every layout.
template <bool BF16>
struct OperandType {
  typedef bf16_x8 type;
};
template <>
struct OperandType<false> {
  typedef f32_x8 type;
};
template <bool BF16>
using Operand = typename OperandType<BF16>::type;

// c += a . b^T; element r of lane l of the 32 x 32 result is row
// 8 (r / 4) + 4 (l / 32) + r % 4 (a's), column l % 32 (b's).
template <bool BF16>
__device__ __forceinline__ void multiply(f32_x16& c, const Operand<BF16>& a, const Operand<BF16>& b) {
#if defined(__HIP_DEVICE_COMPILE__)
  if constexpr (BF16) {
    c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[j], b[j], c, 0, 0, 0);
  }
#endif
}

// Values 8 step .. 8 step + 7 of a 32 x 32 result as an operand whose row is
// the result's column: its summed axis is the result's rows 16 step .. 16 step
// + 15 in the order 4 h .. 4 h + 3, 8 + 4 h .. 8 + 4 h + 3 for half h, which
// is the order in which column_operand() reads a tile's rows.
template <bool BF16>
__device__ __forceinline__ Operand<BF16> result_operand(const f32_x16& c, int step) {
  if constexpr (BF16) {
    const uint4 w = make_uint4(pack_bf16(c[8 * step], c[8 * step + 1]), pack_bf16(c[8 * step + 2], c[8 * step + 3]),
                               pack_bf16(c[8 * step + 4], c[8 * step + 5]), pack_bf16(c[8 * step + 6], c[8 * step + 7]));
    return __builtin_bit_cast(bf16_x8, w);
  } else {
    Operand<BF16> o;
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = c[8 * step + j];
    return o;
  }
}

// Keeps the compiler from moving instructions across: where an order of reads
// and products was chosen by hand it would undo it, each product then waiting
// for operands that were read just before.
__device__ __forceinline__ void pin() {
#if defined(__HIP_DEVICE_COMPILE__)
  __builtin_amdgcn_sched_barrier(0);
#endif
}

// Row of element r of a 32 x 32 result, without the lane's 4 (l / 32).
constexpr int result_row(int r) { return 8 * (r / 4) + r % 4; }

// ---- Tiles -----------------------------------------------------------------------

// ROWS rows of DP values (heads of up to DP values, the rest zero) in shared
// memory, in chunks of 16 bytes.  Chunk c of row r lies at place c ^ key(r)
// of its row: 16 consecutive rows have their chunk c in 16 different places,
// so the 16 lanes that read operands by rows in one cycle meet all 64 banks, and
// the 4 rows from 4 r on have 2 neighbouring pairs of chunks in 8 different
// places, so the 32 lanes that read them by columns (bf16) do too.  (With the
// pairs of 4 rows apart but not the 2 neighbours', every transposing read took
// twice as long.)
template <bool BF16, int DP, int ROWS>
struct Tile {
  static constexpr int kElem = BF16 ? 2 : 4;
  static constexpr int kPitch = DP * kElem;
  static constexpr int kChunks = kPitch / 16;
  static constexpr int kBytes = ROWS * kPitch;
  __device__ static __forceinline__ int key(int row) {
    if (!BF16) return row & 15;
    const int upper = (row >> 2 & 1) << 1 | (row >> 3 & 1);
    return kChunks == 8 ? (row >> 1 & 1) << 2 | upper : (row & 3) << 2 | upper;  // 8 chunks: two rows meet all banks
  }
};

// Offsets of a lane's operands in a tile, `base` bytes (whole tiles) in; steps
// along the head (kk: 16 values, dt: 32 values) flip chunk bits, steps along the
// rows are constants.
template <bool BF16, int DP>
struct RowOperand {
  typedef Tile<BF16, DP, 32> T;
  uint32_t at;
  __device__ __forceinline__ explicit RowOperand(int lane, int base = 0) {
    const int row = lane & 31, chunk = (lane >> 5) * (BF16 ? 1 : 2);
    at = base + row * T::kPitch + ((chunk ^ T::key(row)) << 4);
  }
  // Rows sub * 32 .. + 31, values 16 kk .. 16 kk + 15.
  __device__ __forceinline__ Operand<BF16> load(const uint8_t* tile, int sub, int kk) const {
    const uint8_t* const p = tile + sub * 32 * T::kPitch;
    if constexpr (BF16) {
      return *reinterpret_cast<const bf16_x8*>(p + (at ^ (kk << 5)));
    } else {
      Operand<BF16> o;
      const float4 a = *reinterpret_cast<const float4*>(p + (at ^ (kk << 6)));
      const float4 b = *reinterpret_cast<const float4*>(p + (at ^ (kk << 6) ^ 16));
      o[0] = a.x, o[1] = a.y, o[2] = a.z, o[3] = a.w;
      o[4] = b.x, o[5] = b.y, o[6] = b.z, o[7] = b.w;
      return o;
    }
  }
};
template <bool BF16, int DP>
struct ColumnOperand {
  typedef Tile<BF16, DP, 32> T;
  static constexpr int kParts = BF16 ? 2 : 8;
  uint32_t at[kParts];
  __device__ __forceinline__ explicit ColumnOperand(int lane, int base = 0) {
    if constexpr (BF16) {
      // A transposing read gives lane i of 16 column i of a block of 4 rows
      // by 16 columns, to whose row i / 4, columns 4 (i % 4) .. + 3 it points.
      const int i = lane & 15, block = lane >> 4;
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int row = 8 * p + 4 * (block >> 1) + (i >> 2), chunk = (block & 1) * 2 + ((i & 3) >> 1);
        at[p] = base + row * T::kPitch + ((chunk ^ T::key(row)) << 4) + ((i & 1) << 3);
      }
    } else {
      const int col = lane & 31;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int row = 4 * (lane >> 5) + (j & 3) + 8 * (j >> 2);
        at[j] = base + row * T::kPitch + (((col >> 2) ^ T::key(row)) << 4) + ((col & 3) << 2);
      }
    }
  }
  // Columns 32 dt .. + 31 as the operand's rows, the tile's rows 16 step ..
  // + 15 as its summed axis.
  __device__ __forceinline__ Operand<BF16> load(const uint8_t* tile, int step, int dt) const {
    Operand<BF16> o{};
#if defined(__HIP_DEVICE_COMPILE__)
    const uint8_t* const p = tile + step * 16 * T::kPitch;
    if constexpr (BF16) {
      const s16_x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_ptr)(p + (at[0] ^ (dt << 6))));
      const s16_x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_ptr)(p + (at[1] ^ (dt << 6))));
      o = __builtin_bit_cast(bf16_x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = *reinterpret_cast<const float*>(p + (at[j] ^ (dt << 7)));
    }
#endif
    return o;
  }
};

// Loads of a tile by WAVES waves, 16 bytes per lane straight into shared
// memory.  Rows past `valid` and values past the head read as zeros: their
// offsets lie outside the buffer (also where rows share memory, stride 0).
template <bool BF16, int DP, int ROWS, int WAVES>
struct TileLoader {
  typedef Tile<BF16, DP, ROWS> T;
  static constexpr int kLoads = T::kBytes / 16 / kWave / WAVES;
  static_assert(kLoads * 16 * kWave * WAVES == T::kBytes, "whole loads");
  uint32_t off[kLoads];
  static constexpr uint32_t kRowsPerLoad = WAVES * kWave / T::kChunks;
  uint32_t row_bytes, head_bytes, first_row;
  int wave;
  __device__ __forceinline__ TileLoader(int wave_, int lane, int64_t row_stride, int head_dim) : wave(wave_) {
    first_row = (wave * kWave + lane) / T::kChunks;
    row_bytes = static_cast<uint32_t>(row_stride * T::kElem);
    head_bytes = static_cast<uint32_t>(head_dim * T::kElem);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int slot = (i * WAVES + wave) * kWave + lane, row = slot / T::kChunks;
      const uint32_t byte = static_cast<uint32_t>(((slot % T::kChunks) ^ T::key(row)) << 4);
      off[i] = byte < head_bytes ? row * row_bytes + byte : 0x80000000u;
    }
  }
#if defined(__HIP_DEVICE_COMPILE__)
  // The tile whose first row is at `first`; rows: of it that exist (at most ROWS; 0 or below: all zeros).
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t source(const uint8_t* first, int rows) const {
    const int bytes = __builtin_amdgcn_readfirstlane(rows > 0 ? static_cast<int>((rows - 1) * row_bytes + head_bytes) : 0);
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(first), 0, bytes, 0x00020000);
  }
  // Load i < kLoads of the tile.
  __device__ __forceinline__ void issue(__amdgpu_buffer_rsrc_t src, int i, int rows, uint8_t* tile) const {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (lds_void_ptr)(tile + 16 * ((i * WAVES + wave) * kWave)), 16,
                                             static_cast<int>(first_row + i * kRowsPerLoad) >= rows ? 0x80000000u : off[i], 0, 0, 0);
  }
#endif
  __device__ __forceinline__ void issue(const uint8_t* first, int64_t valid, uint8_t* tile) const {
#if defined(__HIP_DEVICE_COMPILE__)
    const int rows = __builtin_amdgcn_readfirstlane(valid >= ROWS ? ROWS : valid > 0 ? static_cast<int>(valid) : 0);
    const auto src = source(first, rows);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) issue(src, i, rows, tile);
#endif
  }
};

// This wave's loads into shared memory have landed, all of them or all but
// the N youngest.
template <int N>
__device__ __forceinline__ void wait_loads() {
#if defined(__HIP_DEVICE_COMPILE__)
  // gfx9 encoding: vmcnt in bits 0-3 and 14-15, other counters left open.
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | (N >> 4) << 14);
#endif
}

// The operands of one row of queries (or keys) from memory: lane l takes the
// 8-value pieces of its row that its half l / 32 needs; `row` null: zeros.
template <bool BF16, int DP>
__device__ __forceinline__ void load_row_operands(const uint8_t* row, int head_dim, int half, Operand<BF16> (&o)[DP / 16]) {
#pragma unroll
  for (int kk = 0; kk < DP / 16; ++kk) {
    const int d = 16 * kk + 8 * half;
    if (row && d < head_dim) {
      o[kk] = *reinterpret_cast<const Operand<BF16>*>(row + d * (BF16 ? 2 : 4));
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) o[kk][j] = 0;
    }
  }
}

// Stores the column `lane % 32` of DP / 32 results (rows: the head's values)
// times `scale` as one row of a tensor; null: nothing.
template <bool BF16, int DP>
__device__ __forceinline__ void store_columns(const f32_x16 (&c)[DP / 32], float scale, uint8_t* row, int head_dim, int half) {
#pragma unroll
  for (int dt = 0; dt < DP / 32; ++dt) {
    if constexpr (BF16) {
#pragma unroll
      for (int g = 0; g < 2; ++g) {  // 16 values: two quads here, two in the other half
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          // The lower lanes end with the quads of rows 0-3 and 4-7, the upper ones with 8-11 and 12-15.
          const uint32_t a = pack_bf16(c[dt][8 * g + 2 * i] * scale, c[dt][8 * g + 2 * i + 1] * scale);
          const uint32_t b = pack_bf16(c[dt][8 * g + 4 + 2 * i] * scale, c[dt][8 * g + 5 + 2 * i] * scale);
          const auto ab = __builtin_amdgcn_permlane32_swap(a, b, false, false);
          w[i] = ab[0];
          w[2 + i] = ab[1];
        }
        const int d = 32 * dt + 16 * g + 8 * half;
        if (row && d < head_dim) *reinterpret_cast<uint4*>(row + 2 * d) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    } else {
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int d = 32 * dt + 8 * g + 4 * half;
        if (row && d < head_dim)
          *reinterpret_cast<float4*>(row + 4 * d) =
              make_float4(c[dt][4 * g] * scale, c[dt][4 * g + 1] * scale, c[dt][4 * g + 2] * scale, c[dt][4 * g + 3] * scale);
      }
    }
  }
}

// v of this lane and of lane ^ 32.
__device__ __forceinline__ void both_halves(float v, float* a, float* b) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  const auto ab = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const uint32_t x = ab[0], y = ab[1];
  *a = __builtin_bit_cast(float, x);
  *b = __builtin_bit_cast(float, y);
}

}  // namespace cq
