// Embedding lookup with scaling, from floating-point rows or straight from CQ
// storage, and the gradient of the table by sorted tokens.
//
// Lookup: out[i] = scale * W[token i].  From CQ storage a row is decoded as
// dequantization decodes it ("Cactus Quants CQ2-bit Quantization: Extreme
// Compression for Edge LLMs", section The CQ2-bit Implementation Pipeline):
// (norm / G) H levels[idx] per group, H the +-1 Sylvester matrix, in one pass
// from packed bytes to scaled output.  A lane owns 16 bytes of output (4
// float32 or 8 bf16 columns), so a wave's store instruction writes whole
// kilobytes; a group lies over G / 4 or G / 8 lanes, its first butterfly
// stages inside a lane and the rest between lanes (lanes.h).
//
// Gradient: grad[v] = scale * sum of dout[i] over the positions i with
// token i = v.  The positions are sorted by token (a stable radix sort); then
// the sorted list is cut into pieces of 16, 32 or 64 positions by its length,
// and a wave streams the rows of dout of one piece over 256
// columns, writing a table row where a token's run ends: no atomics, and no
// order that changes between runs: position order within a piece.  Runs longer
// than a piece leave one sum per piece, which are added afterwards in four
// consecutive shares and these in order.  The rows of absent tokens,
// most of the bytes at training sizes, are cleared by a plain fill that runs
// beside the sort.  Short lists are not sorted: one launch compares every
// position with all others (below).
// 16384 bf16 rows of 4096 into 32000 rows of float32 (0.66 GB): 91 us for the
// fill with the sort beside it, 56 for the sums, 9 to join long runs, 4.2 TB/s
// over all; a block per table row that searched the sorted list for its run,
// zeros included, took 250.  With cached instead of streaming stores the fill
// takes 75 us and the sums, behind its write-backs, 76.
#include <utility>

#include "lanes.h"

namespace cq {
namespace {

constexpr int kBlock = 256;
constexpr int kWaves = kBlock / kWave;

__device__ __forceinline__ int64_t token_at(const void* tokens, int bytes, int64_t i) {
  return bytes == 8 ? static_cast<const int64_t*>(tokens)[i] : static_cast<const int32_t*>(tokens)[i];
}

// Lookups of 16 MiB and more leave with streaming stores (and from CQ storage
// several units to a wave).  Rows of 4096, cached and streaming, us: from 2
// bits to bf16 8 MiB 5.7 and 6.2, 16 MiB 9.0 and 8.4, 64 MiB 22.6 and 16.2; to
// float32 8 MiB 5.3 and 5.4, 16 MiB 8.1 and 7.4, 64 MiB 20.8 and 13.2; bf16
// rows 8 MiB 4.0 and 4.0, 16 MiB 5.8 and 4.9, 32 MiB 11.6 and 10.3.  Smaller
// ones stay in the caches for what reads them.
constexpr int64_t kStreamBytes = int64_t(16) << 20;

// E consecutive output columns from column c of a row of dim columns; WIDE:
// rows start on and hold whole 16-byte pieces.
template <bool BF16, int E, bool WIDE, bool STREAM>
__device__ __forceinline__ void store_columns(uint8_t* row, int64_t c, int64_t dim, const float (&v)[E]) {
  if constexpr (WIDE) {
    if (c >= dim) return;
    constexpr int V = Piece<BF16>::kElems;
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    u32x4* o = reinterpret_cast<u32x4*>(row + c * Piece<BF16>::kBytes);
#pragma unroll
    for (int i = 0; i < E / V; ++i) {
      const u32x4 u = __builtin_bit_cast(u32x4, pack_piece<BF16>(v + i * V));
      if constexpr (STREAM)
        __builtin_nontemporal_store(u, o + i);
      else
        o[i] = u;
    }
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (c + i < dim) store_elem<BF16>(row, c + i, v[i]);
  }
}

// ---- Dense lookup -----------------------------------------------------------------

// One wave per unit: 64 E columns of one token's row, E = 8 when either type
// is bf16, else 4.
template <bool IN16, bool OUT16, bool WIDE, bool STREAM>
__global__ void __launch_bounds__(kBlock)
embed_kernel(EmbedArgs a, uint32_t units, uint32_t per_row) {
  constexpr int E = IN16 || OUT16 ? 8 : 4, V = Piece<IN16>::kElems;
  const int lane = threadIdx.x & (kWave - 1);
  const uint32_t u = blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  if (u >= units) return;
  const uint32_t i = u / per_row;
  const int64_t c = static_cast<int64_t>((u - i * per_row) * kWave + lane) * E;
  const int64_t tok = token_at(a.tokens, a.token_bytes, i);
  const bool in = tok >= 0 && tok < a.vocab;
  float v[E];
  if (in) {
    const uint8_t* row = a.table + tok * a.dim * Piece<IN16>::kBytes;
    if constexpr (WIDE) {
      const int64_t cc = c < a.dim ? c : 0;
#pragma unroll
      for (int k = 0; k < E / V; ++k)
        unpack_piece<IN16>(reinterpret_cast<const uint4*>(row + cc * Piece<IN16>::kBytes)[k], v + k * V);
    } else {
#pragma unroll
      for (int k = 0; k < E; ++k) v[k] = load_elem<IN16>(row, c + k < a.dim ? c + k : 0);
    }
#pragma unroll
    for (int k = 0; k < E; ++k) v[k] *= a.scale;
  } else {
#pragma unroll
    for (int k = 0; k < E; ++k) v[k] = 0.0f;
  }
  store_columns<OUT16, E, WIDE, STREAM>(a.out + i * a.dim * Piece<OUT16>::kBytes, c, a.dim, v);
}

// ---- Lookup from CQ storage ----------------------------------------------------------

// The E codes of columns `within` .. of a group at p (gbytes long), as bit
// fields from bit 0 (trit storage: 2-bit fields).
template <int SB, int E>
__device__ __forceinline__ uint32_t load_codes(const uint8_t* p, int within, int gbytes, const uint16_t* trits) {
  if constexpr (SB == kTritStorage) {
    const int b = within / 5, last = gbytes - 1;
    uint32_t f = trits[p[b]] | (static_cast<uint32_t>(trits[p[b + 1 < last ? b + 1 : last]]) << 10);
    if constexpr (E == 8) f |= static_cast<uint32_t>(trits[p[b + 2 < last ? b + 2 : last]]) << 20;
    return f >> (2 * (within - 5 * b));
  } else if constexpr (SB == 3) {
    const uint8_t* b = p + (within * 3) / 8;
    if constexpr (E == 8) return b[0] | (b[1] << 8) | (static_cast<uint32_t>(b[2]) << 16);
    return (b[0] | (b[1] << 8)) >> ((within * 3) & 7);
  } else {
    const uint8_t* b = p + (within * SB) / 8;
    if constexpr (SB * E == 8) return *b;
    if constexpr (SB * E == 16) return *reinterpret_cast<const uint16_t*>(b);
    return *reinterpret_cast<const uint32_t*>(b);
  }
}

// P units of 64 E columns of one row per wave, their loads issued together
// (P = 4 for large lookups: 2 and 8 were no faster); per_row: waves per row.
template <int SB, bool OUT16, bool WIDE, int P>
__global__ void __launch_bounds__(kBlock)
embed_packed_kernel(EmbedArgs a, LevelTable lv, uint32_t waves, uint32_t per_row) {
  constexpr int E = OUT16 ? 8 : 4;
  constexpr int FB = SB == kTritStorage ? 2 : SB;
  __shared__ float tab[kMaxLevels];  // 16 banks: any mix of codes reads without conflict
  __shared__ uint16_t trits[SB == kTritStorage ? 256 : 1];
  if (threadIdx.x < kMaxLevels) {
    const float l = level_at(lv, threadIdx.x);
    tab[threadIdx.x] = l;
    wait_lds_writes();
    hold_value(l);
  }
  if constexpr (SB == kTritStorage) {
    const uint32_t f = trit_table_entry(threadIdx.x);
    trits[threadIdx.x] = static_cast<uint16_t>(f);
    wait_lds_writes();
    hold_value(f);
  }
  __syncthreads();
  const int lane = threadIdx.x & (kWave - 1), label = lane_label(lane);
  const uint32_t w = blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  if (w >= waves) return;
  const uint32_t i = w / per_row;
  const int64_t first = static_cast<int64_t>(w - i * per_row) * (P * kWave * E) + label * E;  // this lane's columns
  const int64_t tok = token_at(a.tokens, a.token_bytes, i);
  const bool in = tok >= 0 && tok < a.vocab;
  const int shift = __builtin_ctz(a.group);
  const int64_t ngr = (a.dim + a.group - 1) >> shift;
  const uint8_t* const packed = a.packed + (in ? tok : 0) * ngr * a.gbytes;
  const uint16_t* const norms = a.norms + (in ? tok : 0) * ngr;
  uint32_t raw[P];
  float f[P];
#pragma unroll
  for (int j = 0; j < P; ++j) {
    raw[j] = 0;
    f[j] = 0.0f;
    if (in) {  // a token outside the table has norms of zero
      const int64_t c = first + j * (kWave * E), g = c >> shift;
      const int64_t gc = g < ngr ? g : 0;
      raw[j] = load_codes<SB, E>(packed + gc * a.gbytes, static_cast<int>(c & (a.group - 1)), a.gbytes, trits);
      f[j] = static_cast<float>(__builtin_bit_cast(_Float16, norms[gc]));
    }
  }
  const float unit = label_sign(label, a.group / E) * a.scale / static_cast<float>(a.group);
  uint8_t* const out = a.out + i * a.dim * Piece<OUT16>::kBytes;
#pragma unroll
  for (int j = 0; j < P; ++j) {
    float y[E];
#pragma unroll
    for (int k = 0; k < E; ++k) y[k] = tab[(raw[j] >> (FB * k)) & ((1u << FB) - 1u)];
    lane_butterfly(y);
    label_butterfly(y, label, a.group / E);
    const float s = f[j] * unit;
#pragma unroll
    for (int k = 0; k < E; ++k) y[k] *= s;
    store_columns<OUT16, E, WIDE, (P > 1)>(out, first + j * (kWave * E), a.dim, y);
  }
}

// ---- Gradient: sorting the positions by token --------------------------------------------

constexpr int kDigit = 256;       // 8-bit digits, least significant first
// Tokens and vocabulary that one launch sorts, the fill running beside it: two
// passes in one block took 32.6 us for 12000 tokens of 1000, four launches over
// tiles 24 and their gaps, ranges take 17.1 (6000 of 4000: 18.4, 23 and 9.7).
// 2^14 tokens are what a range's list in shared memory holds (64 KiB).  Past
// 2^18 rows there are so many ranges, each reading all tokens, that tiles are
// faster, first with many tokens.  Whole calls, ranges and tiles, us, 3000, 8192 and 16384 bf16 rows of 64 into 128256 rows 24.1 and
// 45.9, 26.7 and 49.2, 42.5 and 55.3; into 256000 31.9 and 50.7, 38.7 and 54.6,
// 60.8 and 58.4; into 524288 52.5 and 62.6, 62.2 and 65.3, 103.5 and 71.2; into
// 2^20 88.4 and 86.6, 108 and 89.6, 179 and 94.4 (rows of 512 into 524288 228
// and 217, 244 and 220, 268 and 228).
constexpr int64_t kSortOne = 16384, kSortVocab = int64_t(1) << 18;
bool one_launch_sorts(int64_t n, int64_t vocab) { return n <= kSortOne && vocab <= kSortVocab; }

// A constant in a register of its own, so that hold_value() holds that one.
__device__ __forceinline__ uint32_t in_register(uint32_t v) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("" : "+v"(v));
#endif
  return v;
}

// Sort key: the token, or vocab (past every row) where it is outside the table.
__device__ __forceinline__ uint32_t token_key(const EmbedGradArgs& a, int64_t i) {
  const int64_t t = token_at(a.tokens, a.token_bytes, i);
  return static_cast<uint32_t>(t >= 0 && t < a.vocab ? t : a.vocab);
}

// Lanes of the wave whose digit equals this lane's.
__device__ __forceinline__ uint64_t same_digit(uint32_t d) {
  uint64_t m = ~0ull;
#pragma unroll
  for (int b = 0; b < 8; ++b) {
    const bool one = (d >> b) & 1u;
    const uint64_t v = __ballot(one);
    m &= one ? v : ~v;
  }
  return m;
}

// Ranks a wave's keys digit by digit in order: rank = keys of the same digit
// seen before by this wave.  hist: the wave's 256 counters in LDS, zeroed.
// volatile: other lanes of the wave change them between steps (the LDS serves
// a wave's operations in order).
template <int IPT>
__device__ __forceinline__ void rank_keys(const uint32_t (&key)[IPT], int shift, volatile uint32_t* hist,
                                          uint32_t (&rank)[IPT]) {
  const int lane = threadIdx.x & (kWave - 1);
#pragma unroll
  for (int i = 0; i < IPT; ++i) {
    const uint32_t d = (key[i] >> shift) & (kDigit - 1);
    const uint64_t m = same_digit(d);
    const uint32_t below = __popcll(m & ((1ull << lane) - 1ull));
    const uint32_t base = hist[d];
    rank[i] = base + below;
    const uint32_t next = base + static_cast<uint32_t>(__popcll(m));
    if (below == 0) hist[d] = next;
    wait_lds_writes();
    hold_value(next);
  }
}

// Exclusive sum over the first 256 threads' values (one per digit).
__device__ __forceinline__ uint32_t digit_scan(uint32_t v, uint32_t* part) {
  const int t = threadIdx.x, lane = t & (kWave - 1);
  uint32_t x = v;
#pragma unroll
  for (int h = 1; h < kWave; h <<= 1) {
    const uint32_t o = __shfl_up(x, h, kWave);
    if (lane >= h) x += o;
  }
  if (t < kDigit && lane == kWave - 1) {
    part[t / kWave] = x;
  }
  wait_lds_writes();
  hold_value(x);
  __syncthreads();
  uint32_t before = 0;
  if (t < kDigit)
    for (int w = 0; w < t / kWave; ++w) before += part[w];
  return before + x - v;
}

// Zeros over the gradient by block `block` of `blocks`, in contiguous pieces
// of 64 bytes per thread.
constexpr int kClearBytes = 64;
constexpr int64_t kMaxClear = int64_t(1) << 23;  // blocks; more bytes than they hold take turns
__device__ __forceinline__ void clear_grad(const EmbedGradArgs& a, int64_t block, int64_t blocks) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  const int64_t bytes = a.vocab * a.dim * (a.grad_bf16 ? 2 : 4), whole = bytes / 16, each = blockDim.x * (kClearBytes / 16);
  u32x4* const to = reinterpret_cast<u32x4*>(a.grad);
  for (int64_t first = block * each; first < whole; first += blocks * each) {
#pragma unroll
    for (int k = 0; k < kClearBytes / 16; ++k) {
      const int64_t i = first + k * static_cast<int64_t>(blockDim.x) + threadIdx.x;
      if (i < whole) __builtin_nontemporal_store(u32x4{0, 0, 0, 0}, to + i);
    }
  }
  if (block == 0 && threadIdx.x < bytes % 16 / 2) reinterpret_cast<uint16_t*>(to + whole)[threadIdx.x] = 0;
}
// Blocks of `threads` threads that clear all of it, at most `most` (none when
// accumulating).
uint32_t clear_blocks(const EmbedGradArgs& a, int threads, int64_t most) {
  const int64_t bytes = a.accumulate ? 0 : a.vocab * a.dim * (a.grad_bf16 ? 2 : 4), each = threads * kClearBytes;
  const int64_t want = (bytes + each - 1) / each;
  return static_cast<uint32_t>(want < most ? want : most);
}

// The whole sort in one launch: block b takes the keys 256 b .. 256 b + 255
// out of all n, which tells it where they go (the smaller keys' number) and
// their order of position, and sorts them by their last digit: counts per wave,
// then ranks.  The launch's other blocks clear the gradient.  IPT: tokens per
// lane, a wave's 64 IPT consecutive.
constexpr int kOneThreads = 1024, kOneWaves = kOneThreads / kWave;
template <int IPT>
__global__ void __launch_bounds__(kOneThreads)
sort_ranges_kernel(EmbedGradArgs a, uint32_t ranges, uint32_t* __restrict__ keys, uint32_t* __restrict__ order) {
  __shared__ uint32_t hist[kOneWaves][kDigit];
  __shared__ uint32_t part[kDigit / kWave];
  __shared__ uint32_t smaller[kOneWaves], inside[kOneWaves];
  __shared__ uint32_t list[kOneThreads * IPT];  // digit and position of the range's keys, by position
  if (blockIdx.x >= ranges) return clear_grad(a, blockIdx.x - ranges, gridDim.x - ranges);
  const int t = threadIdx.x, lane = t & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(t / kWave);
  const uint32_t n = static_cast<uint32_t>(a.n), lo = blockIdx.x * kDigit;
  const uint32_t first = wave * kWave * IPT + lane;
  uint32_t key[IPT];
#pragma unroll
  for (int i = 0; i < IPT; ++i) {
    const uint32_t p = first + i * kWave;
    key[i] = p < n ? token_key(a, p) : 0xFFFFFFFFu;
  }
  uint32_t under = 0, mine = 0;
#pragma unroll
  for (int i = 0; i < IPT; ++i) {
    under += __popcll(__ballot(key[i] < lo));
    mine += __popcll(__ballot(key[i] - lo < kDigit));
  }
  const uint32_t zero = in_register(0);
  for (int i = t; i < kOneWaves * kDigit; i += kOneThreads) hist[i / kDigit][i % kDigit] = zero;
  const uint32_t u = in_register(under), v = in_register(mine);
  if (lane == 0) {
    smaller[wave] = u;
    inside[wave] = v;
  }
  wait_lds_writes();
  hold_values(zero, u, v);
  __syncthreads();
  uint32_t base = 0, at = 0, count = 0;
  for (int w = 0; w < kOneWaves; ++w) {
    base += smaller[w];
    at += w < wave ? inside[w] : 0;
    count += inside[w];
  }
  if (count == 0) return;  // the same for the block
#pragma unroll
  for (int i = 0; i < IPT; ++i) {
    const bool in = key[i] - lo < kDigit;
    const uint64_t m = __ballot(in);
    const uint32_t item = (key[i] - lo) << 16 | (first + i * kWave);
    if (in) list[at + __popcll(m & ((1ull << lane) - 1ull))] = item;
    wait_lds_writes();
    hold_value(item);
    at += __popcll(m);
  }
  __syncthreads();
  // A wave ranks consecutive items.
  const uint32_t share = (count + kOneThreads - 1) / kOneThreads * kWave, begin = wave * share;
  volatile uint32_t* const mine_of = hist[wave];  // volatile: other lanes change it between steps
  for (uint32_t p0 = begin; p0 < begin + share && p0 < count; p0 += kWave) {
    const bool in = p0 + lane < count;
    const uint32_t d = list[in ? p0 + lane : p0] >> 16;
    const uint64_t m = same_digit(d) & __ballot(in);
    const uint32_t next = mine_of[d] + static_cast<uint32_t>(__popcll(m));
    if (in && (m & ((1ull << lane) - 1ull)) == 0) mine_of[d] = next;
    wait_lds_writes();
    hold_value(next);
  }
  __syncthreads();
  uint32_t total = 0;
  if (t < kDigit) {
    for (int w = 0; w < kOneWaves; ++w) total += hist[w][t];
  }
  uint32_t run = base + digit_scan(total, part);
  if (t < kDigit) {
    for (int w = 0; w < kOneWaves; ++w) {
      const uint32_t here = run;
      run += hist[w][t];
      hist[w][t] = here;
      wait_lds_writes();
      hold_value(here);
    }
  }
  __syncthreads();
  for (uint32_t p0 = begin; p0 < begin + share && p0 < count; p0 += kWave) {
    const bool in = p0 + lane < count;
    const uint32_t item = list[in ? p0 + lane : p0], d = item >> 16;
    const uint64_t m = same_digit(d) & __ballot(in);
    const uint32_t below = __popcll(m & ((1ull << lane) - 1ull));
    const uint32_t from = mine_of[d], next = from + static_cast<uint32_t>(__popcll(m));
    if (in) {
      if (below == 0) mine_of[d] = next;
      keys[from + below] = lo + d;
      order[from + below] = item & 0xFFFFu;
    }
    wait_lds_writes();
    hold_value(next);
  }
}

// One pass of the many-block sort.  count_kernel leaves every tile's digit
// counts in counts[tile][256]; scatter_kernel adds the counts of smaller
// digits and of earlier tiles itself (tiles * 1 KiB from the L2; a tile's own
// keys and positions are 16 KiB) and moves its tile's keys.  That saves a
// launch per pass and grows with the square of the tiles: whole calls on rows
// of 4 into 32000 rows take 64 us for 2^17 tokens, 80 for 2^18, 194 for 2^20,
// 854 for 2^22 and 2038 for 2^23.
constexpr int kTileIpt = 8, kSortTile = kTileIpt * kBlock;  // 2048 keys per block

__device__ __forceinline__ void tile_keys(const EmbedGradArgs& a, const uint32_t* keys, const uint32_t* order,
                                          uint32_t (&key)[kTileIpt], uint32_t (&pos)[kTileIpt]) {
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
#pragma unroll
  for (int i = 0; i < kTileIpt; ++i) {
    const int64_t p = static_cast<int64_t>(blockIdx.x) * kSortTile + (wave * kTileIpt + i) * kWave + lane;
    const bool in = p < a.n;
    const int64_t pc = in ? p : 0;
    key[i] = keys ? keys[pc] : token_key(a, pc);
    pos[i] = order ? order[pc] : static_cast<uint32_t>(pc);
    if (!in) key[i] = 0xFFFFFFFFu;
  }
}

__global__ void __launch_bounds__(kBlock)
count_kernel(EmbedGradArgs a, int shift, const uint32_t* __restrict__ keys, uint32_t* __restrict__ counts, uint32_t tiles) {
  __shared__ uint32_t hist[kDigit];
  if (blockIdx.x >= tiles) return clear_grad(a, blockIdx.x - tiles, gridDim.x - tiles);
  const uint32_t zero = 0;
  hist[threadIdx.x] = zero;
  wait_lds_writes();
  hold_value(zero);
  __syncthreads();
  uint32_t key[kTileIpt], pos[kTileIpt];
  tile_keys(a, keys, nullptr, key, pos);
  const uint32_t one = 1;
#pragma unroll
  for (int i = 0; i < kTileIpt; ++i) atomicAdd(&hist[(key[i] >> shift) & (kDigit - 1)], one);
  wait_lds_writes();
  hold_value(one);
  __syncthreads();
  counts[static_cast<int64_t>(blockIdx.x) * kDigit + threadIdx.x] = hist[threadIdx.x];
}

__global__ void __launch_bounds__(kBlock)
scatter_kernel(EmbedGradArgs a, int shift, const uint32_t* __restrict__ counts, const uint32_t* __restrict__ keys,
               const uint32_t* __restrict__ order, uint32_t* __restrict__ keys_out, uint32_t* __restrict__ order_out) {
  __shared__ uint32_t hist[kWaves][kDigit];
  __shared__ uint32_t part[kDigit / kWave];
  const int t = threadIdx.x, wave = t / kWave;
  const uint32_t zero = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) hist[w][t] = zero;
  wait_lds_writes();
  hold_value(zero);
  __syncthreads();
  uint32_t key[kTileIpt], pos[kTileIpt], rank[kTileIpt];
  tile_keys(a, keys, order, key, pos);
  rank_keys<kTileIpt>(key, shift, hist[wave], rank);
  uint32_t before = 0, total = 0;  // of digit t: in earlier tiles, in all
#pragma unroll 8
  for (uint32_t b = 0; b < gridDim.x; ++b) {
    const uint32_t c = counts[static_cast<int64_t>(b) * kDigit + t];
    before += b < blockIdx.x ? c : 0u;
    total += c;
  }
  __syncthreads();
  uint32_t run = digit_scan(total, part) + before;
  uint32_t at[kWaves];
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    at[w] = run;
    run += hist[w][t];
  }
#pragma unroll
  for (int w = 0; w < kWaves; ++w) hist[w][t] = at[w];
  wait_lds_writes();
#pragma unroll
  for (int w = 0; w < kWaves; ++w) hold_value(at[w]);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kTileIpt; ++i) {
    const uint32_t to = rank[i] + hist[wave][(key[i] >> shift) & (kDigit - 1)];
    // Slots past n (only the last tile has them) carry the largest key: they
    // rank last and land past n.
    if (to < a.n) {
      keys_out[to] = key[i];
      order_out[to] = pos[i];
    }
  }
}

// ---- Gradient: the sums -------------------------------------------------------------

constexpr int kSlice = 256;    // columns per wave: four per lane

// First sorted index whose key is at least v.
__device__ __forceinline__ uint32_t lower_bound(const uint32_t* __restrict__ keys, uint32_t n, uint32_t v) {
  uint32_t lo = 0, len = n;
  while (len > 0) {
    const uint32_t half = len / 2;
    const bool right = keys[lo + half] < v;
    lo = right ? lo + half + 1 : lo;
    len = right ? len - half - 1 : half;
  }
  return lo;
}

// The runs of equal keys that meet piece c, positions lo .. lo + count - 1.
template <int PIECE>
struct Runs {
  uint32_t lo, count, key;  // key: of position lo + lane
  uint64_t starts;          // bit l: a run starts at position lo + l
  uint32_t head;            // positions of a run that began in an earlier piece
  bool head_long;           // that run is longer than a piece
  uint32_t last;            // where the last run that starts here starts (PIECE: none starts here)
  uint32_t beyond;          // its positions past the piece, at most PIECE
  bool last_long;           // it is longer than a piece
};
template <int PIECE>
__device__ __forceinline__ Runs<PIECE> find_runs(const uint32_t* __restrict__ keys, uint32_t n, uint32_t c, int lane) {
  Runs<PIECE> r;
  r.lo = c * PIECE;
  r.count = n - r.lo < PIECE ? n - r.lo : PIECE;
  const uint32_t none = 0xFFFFFFFFu;  // no key
  const bool here = lane < static_cast<int>(r.count);
  r.key = keys[here ? r.lo + lane : r.lo];
  const uint32_t before = c > 0 && lane < PIECE ? keys[r.lo - PIECE + lane] : none;  // a piece back
  const uint32_t after = lane < PIECE && r.lo + PIECE + lane < n ? keys[r.lo + PIECE + lane] : none;
  const uint32_t left = __shfl_up(r.key, 1, kWave), edge = __builtin_amdgcn_readlane(before, PIECE - 1);
  r.starts = __ballot(here && r.key != (lane == 0 ? edge : left));
  const uint32_t first = r.starts ? static_cast<uint32_t>(__builtin_ctzll(r.starts)) : r.count;
  r.head = first;
  // A run that began earlier and whose last position here is l is longer than
  // a piece if the position PIECE before l is its own too.
  r.head_long = first > 0 && __builtin_amdgcn_readlane(before, first - 1) == __builtin_amdgcn_readlane(r.key, first - 1);
  r.last = r.starts ? 63 - static_cast<uint32_t>(__builtin_clzll(r.starts)) : PIECE;
  const uint32_t tail = __builtin_amdgcn_readlane(r.key, r.count - 1);
  const uint64_t differs = __ballot(after != tail);  // lanes past the piece hold no key: set where PIECE < 64
  r.beyond = differs ? static_cast<uint32_t>(__builtin_ctzll(differs)) : 64;
  r.last_long = r.starts && r.count - r.last + r.beyond > PIECE;
  return r;
}

// Four columns of lane `lane` in slice s: consecutive (WIDE), or 64 apart.
template <bool WIDE>
__device__ __forceinline__ int64_t slice_column(int64_t s, int lane, int k) {
  return s * kSlice + (WIDE ? lane * 4 + k : k * kWave + lane);
}

template <bool BF16, bool WIDE>
__device__ __forceinline__ void load_four(const uint8_t* row, int64_t s, int lane, int64_t dim, float (&v)[4]) {
  if constexpr (WIDE) {
    const int64_t c = slice_column<WIDE>(s, lane, 0), cc = c < dim ? c : 0;
    if constexpr (BF16) {
      const uint2 u = *reinterpret_cast<const uint2*>(row + cc * 2);
      v[0] = bf16_low(u.x);
      v[1] = bf16_high(u.x);
      v[2] = bf16_low(u.y);
      v[3] = bf16_high(u.y);
    } else {
      unpack_piece<false>(*reinterpret_cast<const uint4*>(row + cc * 4), v);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t c = slice_column<WIDE>(s, lane, k);
      v[k] = load_elem<BF16>(row, c < dim ? c : 0);
    }
  }
}

template <bool WIDE>
__device__ __forceinline__ void store_four(uint8_t* row, bool bf16, int64_t s, int lane, int64_t dim,
                                           const float (&v)[4]) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  if constexpr (WIDE) {
    const int64_t c = slice_column<WIDE>(s, lane, 0);
    if (c >= dim) return;
    if (bf16) {
      __builtin_nontemporal_store(u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])},
                                  reinterpret_cast<u32x2*>(row + c * 2));
    } else {
      const uint4 p = pack_piece<false>(v);
      __builtin_nontemporal_store(u32x4{p.x, p.y, p.z, p.w}, reinterpret_cast<u32x4*>(row + c * 4));
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t c = slice_column<WIDE>(s, lane, k);
      if (c >= dim) continue;
      if (bf16)
        store_elem<true>(row, c, v[k]);
      else
        store_elem<false>(row, c, v[k]);
    }
  }
}

// Scaled sum into grad row v (added to it when accumulating).
template <bool WIDE>
__device__ __forceinline__ void put_row(const EmbedGradArgs& a, int64_t v, int64_t s, int lane, float (&acc)[4]) {
  uint8_t* row = a.grad + v * a.dim * (a.grad_bf16 ? 2 : 4);
  float old[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (a.accumulate) {
    if (a.grad_bf16)
      load_four<true, WIDE>(row, s, lane, a.dim, old);
    else
      load_four<false, WIDE>(row, s, lane, a.dim, old);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) acc[k] = a.accumulate ? __builtin_fmaf(acc[k], a.scale, old[k]) : acc[k] * a.scale;
  store_four<WIDE>(row, a.grad_bf16, s, lane, a.dim, acc);
}

// Piece c over 1024 columns, 256 per wave: the rows of dout in sorted order,
// eight in flight, added into acc; where a run ends, its sum goes to its row,
// or for a run longer than a piece to partial slot 2c (a run that goes on
// from an earlier piece, or fills this one) or 2c + 1.
template <bool BF16, bool WIDE, int PIECE>
__global__ void __launch_bounds__(kBlock)
embed_grad_kernel(EmbedGradArgs a, const uint32_t* __restrict__ keys, const uint32_t* __restrict__ order,
                  float* __restrict__ partial) {
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const uint32_t n = static_cast<uint32_t>(a.n);
  const int64_t slices = (a.dim + kSlice - 1) / kSlice;
  const uint32_t per = static_cast<uint32_t>((slices + kWaves - 1) / kWaves);
  const uint32_t c = blockIdx.x / per;
  const int64_t s = static_cast<int64_t>(blockIdx.x - c * per) * kWaves + wave;
  if (s >= slices) return;
  const Runs<PIECE> r = find_runs<PIECE>(keys, n, c, lane);
  // Positions from the piece's first that this wave adds, all of them or from
  // the first run that starts here, to the piece's end or that of its last run.
  const uint32_t from = r.head_long ? 0 : r.head;
  const uint32_t to = r.last < PIECE && !r.last_long ? r.count + r.beyond : r.count;
  const uint32_t o0 = lane < static_cast<int>(r.count) ? order[r.lo + lane] : 0;
  const uint32_t o1 = r.lo + PIECE + lane < n ? order[r.lo + PIECE + lane] : 0;
  const int64_t bytes = a.dim * Piece<BF16>::kBytes;
  float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  const uint64_t ends = r.starts >> 1;  // bit l: position l is a run's last
  constexpr int kAhead = 8;
  for (uint32_t l0 = from; l0 < to; l0 += kAhead) {
    float v[kAhead][4];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const uint32_t l = l0 + i < to ? l0 + i : to - 1;
      const uint32_t row = l < PIECE ? __builtin_amdgcn_readlane(o0, l) : __builtin_amdgcn_readlane(o1, l - PIECE);
      load_four<BF16, WIDE>(a.dout + row * bytes, s, lane, a.dim, v[i]);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const uint32_t l = l0 + i;
      if (l >= to) break;
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[k] += v[i][k];
      const bool end = l + 1 == to || (l < PIECE && ((ends >> l) & 1));
      if (!end) continue;
      const uint32_t at = l < r.count ? l : r.count - 1;  // the run's key is the piece's last key past its end
      const uint32_t key = __builtin_amdgcn_readlane(r.key, at);
      if (key < a.vocab) {
        const bool head = at < r.head, whole = head ? r.head_long : at >= r.last && r.last_long;
        if (whole) {
          const int64_t slot = 2 * static_cast<int64_t>(c) + (head || r.last == 0 ? 0 : 1);
          store_four<WIDE>(reinterpret_cast<uint8_t*>(partial + slot * a.dim), false, s, lane, a.dim, acc);
        } else {
          put_row<WIDE>(a, key, s, lane, acc);
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[k] = 0.0f;
    }
  }
}

// Rows of runs longer than a piece: block (c, slice) serves the run that
// begins in piece c, if any; its waves add a quarter of the pieces each, the
// quarters are added in order.
template <bool WIDE, int PIECE>
__global__ void __launch_bounds__(kBlock)
embed_grad_join_kernel(EmbedGradArgs a, const uint32_t* __restrict__ keys, const float* __restrict__ partial) {
  __shared__ float sums[kWaves][kSlice];
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const uint32_t n = static_cast<uint32_t>(a.n);
  const int64_t slices = (a.dim + kSlice - 1) / kSlice;
  const uint32_t c = static_cast<uint32_t>(blockIdx.x / slices);
  const int64_t s = blockIdx.x - c * slices;
  const Runs<PIECE> r = find_runs<PIECE>(keys, n, c, lane);
  const uint32_t key = __builtin_amdgcn_readlane(r.key, r.count - 1);
  if (!r.last_long || key >= a.vocab) return;  // the whole block
  const uint32_t end = __builtin_amdgcn_readfirstlane(lower_bound(keys, n, key + 1));
  const uint32_t pieces = (end - 1) / PIECE - c + 1, quarter = (pieces + kWaves - 1) / kWaves;
  const uint32_t p0 = wave * quarter, p1 = p0 + quarter < pieces ? p0 + quarter : pieces;
  float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (uint32_t p = p0; p < p1; ++p) {
    const int64_t slot = p == 0 && r.last != 0 ? 2 * static_cast<int64_t>(c) + 1 : 2 * static_cast<int64_t>(c + p);
    float v[4];
    load_four<false, WIDE>(reinterpret_cast<const uint8_t*>(partial + slot * a.dim), s, lane, a.dim, v);
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] += v[k];
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) sums[wave][k * kWave + lane] = acc[k];
  wait_lds_writes();
#pragma unroll
  for (int k = 0; k < 4; ++k) hold_value(acc[k]);
  __syncthreads();
  if (wave != 0) return;
#pragma unroll
  for (int w = 1; w < kWaves; ++w)
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] += sums[w][k * kWave + lane];
  put_row<WIDE>(a, key, s, lane, acc);
}

// ---- Gradient of short lists, in one launch ---------------------------------------------

// No sort: block (i, slice) looks at all tokens, stops unless position i is
// the first of its token, and adds that token's rows, each wave those among its
// quarter of the positions, eight in flight; the quarters are added in order.
// The launch's other blocks clear the rows whose tokens are absent, kScanRows
// (fewer for long rows) each, found the same way.
//
// It is bound by latency (tokens, rows, the store) and, past some thousand
// blocks, by the n * n comparisons per slice: up to 2^23 of them in all it is
// faster than the sort with its three launches.  Scan and sort, us, float32
// rows into 8192 rows: 8 of 96 4.8 and 9.6, 256 of 1000 8.1 and 19.3, 777 of
// 1000 11.2 and 20.3, 2048 of 500 (2^23) 12.9 and 23.6, 1024 of 2048 (2^23)
// 22.9 and 25.2, 1024 of 4096 (2^24) 42.5 and 37.0, 2048 of 2048 (2^25) 41.7
// and 26.5.  Sizes cannot tell how often one token comes up: with half of the
// positions one token its rows are one block's, and the sort is faster from
// some 700 positions on (bf16: 256 of 1000 10.3 and 18.8, 777 of 1000 22.8 and
// 20.4, 1448 of 1024 30.4 and 20.8, 2896 of 256 53.7 and 22.7, where distinct
// tokens take 8.6 and 16.7, 12.0 and 17.4, 15.9 and 17.7, 12.6 and 16.1).
constexpr int64_t kScanCompares = int64_t(1) << 23;
constexpr int64_t kScanMost = 2896;  // tokens: the square root of that
constexpr int kScanList = (kScanMost + kBlock - 1) / kBlock * kWave;
constexpr int kScanRows = 64;
constexpr int64_t kScanBytes = 64 << 10;  // of table rows per clearing block

template <bool BF16, bool WIDE>
__global__ void __launch_bounds__(kBlock)
embed_grad_scan_kernel(EmbedGradArgs a, uint32_t sum_blocks, uint32_t slices, uint32_t rows) {
  __shared__ uint32_t found[kWaves][kScanList];
  __shared__ uint32_t count[kWaves], early[kWaves];
  __shared__ float sums[kWaves][kSlice];
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const uint32_t n = static_cast<uint32_t>(a.n);
  if (blockIdx.x >= sum_blocks) {  // the same for the block
    uint32_t* const present = found[0];
    const uint32_t zero = in_register(0), one = in_register(1);
    if (threadIdx.x < kScanRows) present[threadIdx.x] = zero;
    wait_lds_writes();
    hold_value(zero);
    __syncthreads();
    const int64_t first = static_cast<int64_t>(blockIdx.x - sum_blocks) * rows;
    const uint32_t here = static_cast<uint32_t>(a.vocab - first < rows ? a.vocab - first : rows);
    for (uint32_t p = threadIdx.x; p < n; p += kBlock) {
      const int64_t at = token_at(a.tokens, a.token_bytes, p) - first;
      if (at >= 0 && at < here) present[at] = one;
      wait_lds_writes();
      hold_value(one);
    }
    __syncthreads();
    const float none[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (uint32_t r = wave; r < here; r += kWaves) {
      if (__builtin_amdgcn_readfirstlane(present[r])) continue;
      uint8_t* const row = a.grad + (first + r) * a.dim * (a.grad_bf16 ? 2 : 4);
      for (uint32_t s = 0; s < slices; ++s) store_four<WIDE>(row, a.grad_bf16, s, lane, a.dim, none);
    }
    return;
  }
  const uint32_t i = blockIdx.x / slices, s = blockIdx.x - i * slices;
  const int64_t tok = token_at(a.tokens, a.token_bytes, i);
  if (tok < 0 || tok >= a.vocab) return;
  const uint32_t quarter = (n + kBlock - 1) / kBlock * kWave, begin = wave * quarter;
  uint32_t mine = 0, before = 0;
  for (uint32_t p0 = begin; p0 < begin + quarter && p0 < n; p0 += kWave) {
    const uint32_t p = p0 + lane;
    const bool hit = p < n && token_at(a.tokens, a.token_bytes, p < n ? p : i) == tok;
    const uint64_t hits = __ballot(hit);
    if (hit) found[wave][mine + __popcll(hits & ((uint64_t(1) << lane) - 1))] = p;
    wait_lds_writes();
    hold_value(p);
    if (p0 < i) before |= static_cast<uint32_t>(i - p0 >= kWave ? hits != 0 : (hits & ((uint64_t(1) << (i - p0)) - 1)) != 0);
    mine += __popcll(hits);
  }
  if (lane == 0) {
    count[wave] = mine;
    early[wave] = before;
  }
  wait_lds_writes();
  hold_values(mine, before);
  __syncthreads();
  uint32_t total = 0, any = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    total += count[w];
    any |= early[w];
  }
  if (__builtin_amdgcn_readfirstlane(any)) return;  // an earlier position's block serves this token
  const bool alone = __builtin_amdgcn_readfirstlane(total) == 1;
  if (alone && mine == 0) return;
  const int64_t bytes = a.dim * Piece<BF16>::kBytes;
  float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  constexpr int kAhead = 8;
  for (uint32_t l0 = 0; l0 < mine; l0 += kAhead) {
    float v[kAhead][4];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const uint32_t row = __builtin_amdgcn_readfirstlane(found[wave][l0 + k < mine ? l0 + k : mine - 1]);
      load_four<BF16, WIDE>(a.dout + row * bytes, s, lane, a.dim, v[k]);
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {  // all loads are issued before the first sum
      const bool in = l0 + k < mine;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float t = acc[e] + v[k][e];
        acc[e] = in ? t : acc[e];
      }
    }
  }
  if (alone) {
    put_row<WIDE>(a, tok, s, lane, acc);
    return;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) sums[wave][k * kWave + lane] = acc[k];
  wait_lds_writes();
#pragma unroll
  for (int k = 0; k < 4; ++k) hold_value(acc[k]);
  __syncthreads();
  if (wave != 0) return;
#pragma unroll
  for (int w = 1; w < kWaves; ++w)
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] += sums[w][k * kWave + lane];
  put_row<WIDE>(a, tok, s, lane, acc);
}

uint32_t blocks_of(int64_t waves) { return static_cast<uint32_t>((waves + kWaves - 1) / kWaves); }

int64_t align256(int64_t b) { return (b + 255) & ~int64_t(255); }
// Positions per piece: short lists in small pieces, so that enough waves
// stream them, long ones in large ones, which leave fewer sums to join.  Whole
// calls in pieces of 16, 32 and 64, us, bf16 rows: 3000 of 1000 21.7, 26.6 and
// 37.1; 8192 of 1000 27.3, 31.8 and 40.2; 8192 of 4096 127, 125 and 131; 16384
// of 4096 146, 143 and 144; 65536 of 1024 98.9, 90.4 and 94.5; 131072 of 1024
// 145, 128 and 126; with half of the positions one token 8192 of 1000 39.2, 39.4
// and 46.7, 65536 of 1024 160, 123 and 102, 131072 of 1024 272, 197 and 162.
int piece_of(int64_t n) { return n <= 8192 ? 16 : n <= 65536 ? 32 : 64; }
int64_t pieces_of(int64_t n) { return (n + piece_of(n) - 1) / piece_of(n); }

// Table rows per clearing block of a scan, and the scan's blocks.
int64_t scan_rows(const EmbedGradArgs& a) {
  const int64_t fit = kScanBytes / (a.dim * (a.grad_bf16 ? 2 : 4));
  return fit < 1 ? 1 : fit < kScanRows ? fit : kScanRows;
}
int64_t scan_clear_blocks(const EmbedGradArgs& a) {
  const int64_t rows = scan_rows(a);
  return a.accumulate ? 0 : (a.vocab + rows - 1) / rows;
}

// Tables of 2^30 narrow rows would take the clearing blocks past a launch's
// 2^32 threads; the sort's clearing blocks loop.
bool scans(const EmbedGradArgs& a) {
  const int64_t slices = (a.dim + kSlice - 1) / kSlice;
  return a.n > 0 && a.n <= kScanMost && slices <= kScanCompares / (a.n * a.n) &&
         a.n * slices + scan_clear_blocks(a) <= most_blocks(kBlock);
}

// Workspace of the sort: sorted keys and positions (twice in the many-block sort), the
// tiles' digit counts, the pieces' sums.
struct GradSpace {
  int64_t list, counts, partial, total;
};
GradSpace grad_space(int64_t n, int64_t vocab, int64_t dim) {
  GradSpace g;
  g.list = align256(4 * n);
  const bool many = !one_launch_sorts(n, vocab);
  g.counts = many ? align256((n + kSortTile - 1) / kSortTile * kDigit * 4) : 0;
  g.partial = n > piece_of(n) ? align256(2 * pieces_of(n) * dim * 4) : 0;
  g.total = g.list * (many ? 4 : 2) + g.counts + g.partial;
  return g;
}

// launch(args, waves) for all of a lookup's tokens, per_row waves each.
template <typename F>
hipError_t launch_rows(EmbedArgs a, int64_t per_row, F launch) {
  const int64_t most = most_blocks(kBlock) * kWaves / per_row;
  const int64_t row = a.dim * (a.out_bf16 ? 2 : 4);
  for (int64_t left = a.n; left > 0; left -= a.n) {
    a.n = left < most ? left : most;
    launch(a, static_cast<uint32_t>(a.n * per_row));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    a.tokens = static_cast<const uint8_t*>(a.tokens) + a.n * a.token_bytes;
    a.out += a.n * row;
  }
  return hipSuccess;
}

template <int SB, bool OUT16, bool WIDE, int P>
hipError_t launch_packed_units(const EmbedArgs& all, const LevelTable& lv, int64_t units, hipStream_t s) {
  const int64_t per_row = (units + P - 1) / P;
  return launch_rows(all, per_row, [&](const EmbedArgs& a, uint32_t waves) {
    embed_packed_kernel<SB, OUT16, WIDE, P><<<dim3(blocks_of(waves)), dim3(kBlock), 0, s>>>(
        a, lv, waves, static_cast<uint32_t>(per_row));
  });
}

template <int SB, bool OUT16, bool WIDE>
hipError_t launch_packed_at(const EmbedArgs& a, const LevelTable& lv, hipStream_t s) {
  const int64_t units = (a.dim + kWave * (OUT16 ? 8 : 4) - 1) / (kWave * (OUT16 ? 8 : 4));  // per row
  // Few units in all: one per wave, to spread over the CUs.
  if (a.n * a.dim * (OUT16 ? 2 : 4) < kStreamBytes)
    return launch_packed_units<SB, OUT16, WIDE, 1>(a, lv, units, s);
  return launch_packed_units<SB, OUT16, WIDE, 4>(a, lv, units, s);
}

template <int SB>
hipError_t launch_packed_for(const EmbedArgs& a, const LevelTable& lv, hipStream_t s) {
  if (a.out_bf16)
    return a.dim % 8 == 0 ? launch_packed_at<SB, true, true>(a, lv, s) : launch_packed_at<SB, true, false>(a, lv, s);
  return a.dim % 4 == 0 ? launch_packed_at<SB, false, true>(a, lv, s) : launch_packed_at<SB, false, false>(a, lv, s);
}

template <bool IN16, bool OUT16>
hipError_t launch_embed_at(const EmbedArgs& all, hipStream_t s) {
  constexpr int E = IN16 || OUT16 ? 8 : 4;
  const int64_t per_row = (all.dim + kWave * E - 1) / (kWave * E);
  const bool wide = all.dim % E == 0, stream = all.n * all.dim * (OUT16 ? 2 : 4) >= kStreamBytes;
  return launch_rows(all, per_row, [&](const EmbedArgs& a, uint32_t units) {
    const dim3 grid(blocks_of(units)), block(kBlock);
    const uint32_t per = static_cast<uint32_t>(per_row);
    if (wide && stream)
      embed_kernel<IN16, OUT16, true, true><<<grid, block, 0, s>>>(a, units, per);
    else if (wide)
      embed_kernel<IN16, OUT16, true, false><<<grid, block, 0, s>>>(a, units, per);
    else
      embed_kernel<IN16, OUT16, false, false><<<grid, block, 0, s>>>(a, units, per);
  });
}

template <bool BF16>
hipError_t launch_grad_scan(const EmbedGradArgs& a, hipStream_t s) {
  const int64_t slices = (a.dim + kSlice - 1) / kSlice, sums = a.n * slices, rows = scan_rows(a);
  const dim3 grid(static_cast<uint32_t>(sums + scan_clear_blocks(a))), block(kBlock);
  const uint32_t n_sums = static_cast<uint32_t>(sums), n_slices = static_cast<uint32_t>(slices);
  if (a.dim % 4 == 0)
    embed_grad_scan_kernel<BF16, true><<<grid, block, 0, s>>>(a, n_sums, n_slices, static_cast<uint32_t>(rows));
  else
    embed_grad_scan_kernel<BF16, false><<<grid, block, 0, s>>>(a, n_sums, n_slices, static_cast<uint32_t>(rows));
  return hipGetLastError();
}

template <bool WIDE, int PIECE>
hipError_t launch_grad_sums(const EmbedGradArgs& a, const uint32_t* keys, const uint32_t* order, float* partial,
                            hipStream_t s) {
  const int64_t slices = (a.dim + kSlice - 1) / kSlice;
  const dim3 grid(static_cast<uint32_t>(pieces_of(a.n) * ((slices + kWaves - 1) / kWaves)));
  if (a.dout_bf16)
    embed_grad_kernel<true, WIDE, PIECE><<<grid, dim3(kBlock), 0, s>>>(a, keys, order, partial);
  else
    embed_grad_kernel<false, WIDE, PIECE><<<grid, dim3(kBlock), 0, s>>>(a, keys, order, partial);
  if (a.n > PIECE)  // a run may be longer than a piece
    embed_grad_join_kernel<WIDE, PIECE><<<dim3(static_cast<uint32_t>(pieces_of(a.n) * slices)), dim3(kBlock), 0, s>>>(
        a, keys, partial);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_embed(const EmbedArgs& a, hipStream_t s) {
  if (a.table_bf16) return a.out_bf16 ? launch_embed_at<true, true>(a, s) : launch_embed_at<true, false>(a, s);
  return a.out_bf16 ? launch_embed_at<false, true>(a, s) : launch_embed_at<false, false>(a, s);
}

hipError_t launch_embed_packed(const EmbedArgs& a, int storage, const LevelTable& lv, hipStream_t s) {
  if (storage == 2) return launch_packed_for<2>(a, lv, s);
  if (storage == 3) return launch_packed_for<3>(a, lv, s);
  if (storage == 4) return launch_packed_for<4>(a, lv, s);
  return launch_packed_for<kTritStorage>(a, lv, s);
}

int64_t embed_grad_workspace(int64_t n, int64_t vocab, int64_t dim) {
  return grad_space(n, vocab, dim).total;  // also of a list that is scanned: one contract for all lengths
}

int64_t embed_grad_blocks(int64_t n, int64_t dim) { return pieces_of(n) * ((dim + kSlice - 1) / kSlice); }

hipError_t launch_embed_grad(const EmbedGradArgs& a, uint8_t* ws, hipStream_t s) {
  if (a.n == 0) {  // no tiles: the launch is the fill alone (accumulating calls end before)
    count_kernel<<<dim3(clear_blocks(a, kBlock, kMaxClear)), dim3(kBlock), 0, s>>>(a, 0, nullptr, nullptr, 0);
    return hipGetLastError();
  }
  if (scans(a)) return a.dout_bf16 ? launch_grad_scan<true>(a, s) : launch_grad_scan<false>(a, s);
  const GradSpace g = grad_space(a.n, a.vocab, a.dim);
  auto at = [&](int64_t off) { return reinterpret_cast<uint32_t*>(ws + off); };
  uint32_t *keys = at(0), *order = at(g.list);
  float* partial;
  if (one_launch_sorts(a.n, a.vocab)) {
    partial = reinterpret_cast<float*>(at(2 * g.list));
    // One block per CU in all, the clearing ones looping (or one clearing block
    // per CU where the ranges take more than half).  Whole calls with 1, 2 and 4 per CU, us, bf16 rows of 4096 into
    // 32000 rows: 16384 139.7, 142.9 and 143.4, 8192 123.2, 127.5 and 131.2,
    // 4096 112.0, 115.2 and 118.2; 16384 rows of 512 37.8, 37.4 and 36.2.
    const uint32_t ranges = static_cast<uint32_t>(a.vocab / kDigit + 1);
    const int64_t cus = device_cu_count(), beside = ranges <= cus / 2 ? cus - ranges : cus;
    const dim3 grid(ranges + clear_blocks(a, kOneThreads, beside)), block(kOneThreads);
    if (a.n > 8 * kOneThreads)
      sort_ranges_kernel<16><<<grid, block, 0, s>>>(a, ranges, keys, order);
    else if (a.n > 4 * kOneThreads)
      sort_ranges_kernel<8><<<grid, block, 0, s>>>(a, ranges, keys, order);
    else
      sort_ranges_kernel<4><<<grid, block, 0, s>>>(a, ranges, keys, order);
  } else {
    uint32_t *keys2 = at(2 * g.list), *order2 = at(3 * g.list), *counts = at(4 * g.list);
    partial = reinterpret_cast<float*>(at(4 * g.list + g.counts));
    const uint32_t tiles = static_cast<uint32_t>((a.n + kSortTile - 1) / kSortTile);
    const dim3 grid(tiles), block(kBlock);
    int passes = 1;  // keys run from 0 to vocab
    while (passes < 4 && (a.vocab >> (8 * passes))) ++passes;
    const uint32_t *in_keys = nullptr, *in_order = nullptr;  // the first pass reads the tokens
    for (int p = 0; p < passes; ++p) {
      count_kernel<<<dim3(tiles + (p == 0 ? clear_blocks(a, kBlock, kMaxClear) : 0)), block, 0, s>>>(a, 8 * p, in_keys, counts, tiles);
      scatter_kernel<<<grid, block, 0, s>>>(a, 8 * p, counts, in_keys, in_order, keys2, order2);
      in_keys = keys2;
      in_order = order2;
      std::swap(keys, keys2);
      std::swap(order, order2);
    }
    // The last pass wrote what the swap made `keys` and `order`.
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const bool wide = a.dim % 4 == 0;
  if (piece_of(a.n) == 16)
    return wide ? launch_grad_sums<true, 16>(a, keys, order, partial, s) : launch_grad_sums<false, 16>(a, keys, order, partial, s);
  if (piece_of(a.n) == 32)
    return wide ? launch_grad_sums<true, 32>(a, keys, order, partial, s) : launch_grad_sums<false, 32>(a, keys, order, partial, s);
  return wide ? launch_grad_sums<true, 64>(a, keys, order, partial, s) : launch_grad_sums<false, 64>(a, keys, order, partial, s);
}

}  // namespace cq
