// Log probabilities of given tokens under a row of logits, the row's entropy
// and its most probable tokens, and the gradient.
//
// Per row, x = scale * logits, m = max x:
//   s = sum exp(x - m),  lse = m + log s,  logprob = x_t - lse,
//   entropy = -sum p log p = log s - sum exp(x - m) (x - m) / s.
// Gradient, g and h what reaches logprob and entropy, p = exp(x - lse):
//   dlogits_j = scale (g ([j = t] - p_j) - h p_j (x_j - lse + entropy)).
//
// A block reads its row once and keeps it in registers (rows of up to 131072
// bf16 or 65536 float32 values; longer ones are read again by each pass), so the
// maximum, the sums and the search for the top tokens all run on what the first
// read brought.  4096 bf16 rows of 32000: 70 us without and 74 with 20 top tokens for
// 262 MB, 3.7 and 3.5 TB/s, the vector units busy 86 to 92% (some 18 cycles per value, 4 of
// them the exponential); the gradient 86 us for 524 MB, 6.1 TB/s, which memory and
// the last cache bound.
//
// The top tokens, by value and then by lower index: the threads' maxima form
// 64 groups' maxima, whose k-th largest is a floor that at least k values
// reach and, unless values repeat or crowd into few threads, few more do.
// Those go into a list in shared memory and are ranked against each other.
// A list that overflows falls back to one more read of the row per token.
#include "lanes.h"

namespace cq {
namespace {

constexpr int kGroups = 64;  // of threads; as many as there are lanes to rank them
constexpr int kList = 2048;  // candidates in shared memory
static_assert(kMaxTop <= kGroups, "a floor that kMaxTop values reach");

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kNothing = -10000.0f;  // a power of two that is 0 in float32

// The larger of two, NaN if one is.
__device__ __forceinline__ float at_least(float x, float y) { return __builtin_elementwise_maximum(x, y); }

// Floats as integers of the same order: NaN above all, both zeros equal.
constexpr uint32_t kNanOrder = 0xFFFFFFFEu;  // not ~0, so that every key, token 0's too, is below ~0
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x + 0.0f);
  if (x != x) return kNanOrder;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t order) {
  if (order == kNanOrder) return __builtin_nanf("");
  return __builtin_bit_cast(float, order & 0x80000000u ? order & 0x7FFFFFFFu : ~order);
}
// Larger keys come first: by value, then by lower index.  No value has key 0 or ~0.
__device__ __forceinline__ uint64_t key_of(float x, uint32_t index) {
  return static_cast<uint64_t>(order_of(x)) << 32 | (0xFFFFFFFFu - index);
}

// A row in pieces of 16 bytes from the 16-byte boundary at or before its
// start (the tensor starts on a boundary).  Elements outside the row are -inf,
// which no sum sees.  Words past the row's last one lie outside the buffer and
// are not read.
typedef int i32_x4 __attribute__((ext_vector_type(4)));
template <bool BF16>
struct RowPieces {
  static constexpr int V = Piece<BF16>::kElems, kElem = Piece<BF16>::kBytes;
  const uint8_t* start;  // of piece 0
  int before;            // elements of piece 0 before the row
  int vocab;
  __device__ __forceinline__ RowPieces(const uint8_t* row, int64_t vocab_) : vocab(static_cast<int>(vocab_)) {
    before = static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15) / kElem;
    start = row - before * kElem;
  }
  __device__ __forceinline__ int pieces() const { return (vocab + before + V - 1) / V; }
  __device__ __forceinline__ int index(int piece) const { return piece * V - before; }
  __device__ __forceinline__ uint4 load(int piece) const {
    uint4 r{};
#if defined(__HIP_DEVICE_COMPILE__)
    const auto src = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(start), 0, ((before + vocab) * kElem + 3) & ~3, 0x00020000);
    r = __builtin_bit_cast(uint4, static_cast<i32_x4>(__builtin_amdgcn_raw_buffer_load_b128(src, piece * 16, 0, 0)));
#endif
    return r;
  }
  __device__ __forceinline__ uint4 inside(int piece, uint4 r) const {
    const int e = index(piece);
    if (e < 0 || e + V > vocab) {
      float v[V];
      unpack_piece<BF16>(r, v);
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = static_cast<uint32_t>(e + j) < static_cast<uint32_t>(vocab) ? v[j] : -INFINITY;
      r = pack_piece<BF16>(v);
    }
    return r;
  }
};

template <int WAVES, class T, class Op>
__device__ __forceinline__ T over_waves(T v, T* red, Op op) {
  if ((threadIdx.x & (kWave - 1)) == 0) red[threadIdx.x / kWave] = v;
  wait_lds_writes();
  hold_value(v);
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int i = 1; i < WAVES; ++i) v = op(v, red[i]);
  return v;
}
__device__ __forceinline__ uint64_t wave_max64(uint64_t v) {
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const uint64_t o = __shfl_xor(v, d);
    v = v > o ? v : o;
  }
  return v;
}

// R: pieces of a thread kept in registers; 0: the row is read again instead.
template <bool BF16, int NT, int R>
__global__ void __launch_bounds__(NT) logprobs_kernel(LogprobArgs a) {
  constexpr int V = Piece<BF16>::kElems, kElem = Piece<BF16>::kBytes, kWaves = NT / kWave, kTeam = NT / kGroups;
  __shared__ float red[4][kWaves];
  __shared__ uint64_t red64[2][kWaves];
  __shared__ float group_top[kGroups];
  __shared__ uint64_t list[kList];
  __shared__ int listed;
  __shared__ float floor_value;
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int64_t row = blockIdx.x;
  const uint8_t* const logits = a.logits + row * a.row_stride * kElem;
  const RowPieces<BF16> p(logits, a.vocab);

  uint4 held[R ? R : 1];
  if constexpr (R > 0) {
#pragma unroll
    for (int k = 0; k < R; ++k) held[k] = p.load(k * NT + tid);
#pragma unroll
    for (int k = 0; k < R; ++k) held[k] = p.inside(k * NT + tid, held[k]);
  }
  // f(first index, values) for each of this thread's pieces, in ascending order.
  auto each_piece = [&](auto f) __attribute__((always_inline)) {
    if constexpr (R > 0) {
#pragma unroll
      for (int k = 0; k < R; ++k) {
        // Unpacked anew by each pass: the floats of all passes would not fit the registers.
        asm volatile("" : "+v"(held[k].x), "+v"(held[k].y), "+v"(held[k].z), "+v"(held[k].w));
        float v[V];
        unpack_piece<BF16>(held[k], v);
        f(p.index(k * NT + tid), v);
      }
    } else {
      for (int i = tid; i < p.pieces(); i += 4 * NT) {
        uint4 r[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) r[k] = p.load(i + k * NT);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float v[V];
          unpack_piece<BF16>(p.inside(i + k * NT, r[k]), v);
          f(p.index(i + k * NT), v);
        }
      }
    }
  };

  float mine = -INFINITY;
  each_piece([&](int, const float (&v)[V]) {
#pragma unroll
    for (int j = 0; j < V; ++j) mine = fmaxf(mine, v[j]);
  });
  // The team's maximum, then the block's.
  float team = mine;
#pragma unroll
  for (int d = 1; d < kTeam; d <<= 1) team = fmaxf(team, __shfl_xor(team, d));
  if (a.top > 0 && tid % kTeam == 0) {
    group_top[tid / kTeam] = team;
    wait_lds_writes();
    hold_value(team);
  }
  if (tid == 0) {
    const int none = 0;
    listed = none;
    wait_lds_writes();
    hold_value(none);
  }
  float top = team;
#pragma unroll
  for (int d = kTeam; d < kWave; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
  top = over_waves<kWaves>(top, red[0], [](float x, float y) { return fmaxf(x, y); });
  const float ref = top == -INFINITY ? 0.0f : top;  // nothing but -inf: every term is 0

  if (a.top > 0 && tid < kWave) {
    // The a.top-th largest of the 64 groups' maxima.
    const float g = group_top[lane];
    int before = 0;
    for (int i = 0; i < kGroups; ++i) {
      const float o = group_top[i];
      before += o > g || (o == g && i < lane) ? 1 : 0;
    }
    if (before == a.top - 1) {
      floor_value = g;
      wait_lds_writes();
      hold_value(g);
    }
  }
  // In powers of two.  v - ref first, then the factor: against a rounded ref *
  // factor it would be one operation less, but the largest term would not be
  // exactly 1, and a certain token's log probability not 0 (or above it).
  const float factor = a.scale * kLog2e;
  float sum = 0.0f, weighted = 0.0f;
  each_piece([&](int, const float (&v)[V]) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float t = at_least((v[j] - ref) * factor, kNothing);  // -inf: 0 * t has to stay 0
      const float e = __builtin_amdgcn_exp2f(t);
      sum += e;
      weighted = __builtin_fmaf(e, t, weighted);
    }
  });
  sum = wave_sum(sum);
  weighted = wave_sum(weighted);
  if (lane == 0) {
    red[1][tid / kWave] = sum;
    red[2][tid / kWave] = weighted;
  }
  wait_lds_writes();
  hold_value(sum);
  hold_value(weighted);
  __syncthreads();
  sum = red[1][0];
  weighted = red[2][0];
#pragma unroll
  for (int i = 1; i < kWaves; ++i) {
    sum += red[1][i];
    weighted += red[2][i];
  }
  const float log_sum = __builtin_log2f(sum);
  auto log_prob = [&](float v) __attribute__((always_inline)) {
    return sum == 0.0f ? -INFINITY : __builtin_fmaf(v - ref, a.scale, -log_sum * kLn2);
  };
  if (tid == 0) {
    if (a.lse) a.lse[row] = __builtin_fmaf(ref, a.scale, log_sum * kLn2);
    if (a.entropy) a.entropy[row] = sum == 0.0f ? 0.0f : (log_sum - weighted / sum) * kLn2;
    if (a.logprob) {
      const int64_t t = a.token_bytes == 4 ? static_cast<const int32_t*>(a.tokens)[row] : static_cast<const int64_t*>(a.tokens)[row];
      a.logprob[row] = t >= 0 && t < a.vocab ? log_prob(load_elem<BF16>(logits, t)) : 0.0f;
    }
  }
  if (a.top <= 0) return;

  // Values that reach the floor.
  const float least = floor_value;
  each_piece([&](int first, const float (&v)[V]) {
    float piece_top = v[0];
#pragma unroll
    for (int j = 1; j < V; ++j) piece_top = at_least(piece_top, v[j]);
    if (piece_top < least) return;  // nearly all; a NaN is not below
    uint32_t reach = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) reach |= v[j] < least ? 0u : 1u << j;
    for (; reach; reach &= reach - 1) {  // few: read again rather than picked out of registers
      const uint32_t e = first + __builtin_ctz(reach);
      if (e >= static_cast<uint32_t>(p.vocab)) continue;  // outside the row
      const int at = atomicAdd(&listed, 1);
      if (at < kList) {
        const uint64_t key = key_of(load_elem<BF16>(logits, e), e);
        list[at] = key;
        wait_lds_writes();
        hold_value(key);
      }
    }
  });
  __syncthreads();
  auto put = [&](int rank, uint64_t key) __attribute__((always_inline)) {
    a.top_ids[row * a.top + rank] = 0xFFFFFFFFu - static_cast<uint32_t>(key);
    a.top_logprobs[row * a.top + rank] = log_prob(value_of(static_cast<uint32_t>(key >> 32)));
  };
  const int n = listed;
  if (n <= kList) {
    for (int i = tid; i < n; i += NT) {
      const uint64_t key = list[i];
      int rank = 0;
      for (int o = 0; o < n; ++o) rank += list[o] > key ? 1 : 0;
      if (rank < a.top) put(rank, key);
    }
    return;
  }
  uint64_t last = ~0ull;
  for (int rank = 0; rank < a.top; ++rank) {
    uint64_t best = 0;
    for (int i = tid; i < p.pieces(); i += NT) {
      float v[V];
      unpack_piece<BF16>(p.load(i), v);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const uint32_t e = p.index(i) + j;
        const uint64_t key = key_of(v[j], e);
        if (e < static_cast<uint32_t>(p.vocab) && key < last && key > best) best = key;
      }
    }
    best = over_waves<kWaves>(wave_max64(best), red64[rank & 1], [](uint64_t x, uint64_t y) { return x > y ? x : y; });
    if (tid == 0) put(rank, best);
    last = best;
  }
}

// A thread's pieces of a row's gradient.
constexpr int kGradThreads = 256, kGradPieces = 4;

template <bool BF16>
__global__ void __launch_bounds__(kGradThreads) logprobs_grad_kernel(LogprobArgs a, int parts, int blocks) {
  constexpr int V = Piece<BF16>::kElems, kElem = Piece<BF16>::kBytes;
  const int64_t row = blockIdx.x / blocks;
  int part = blockIdx.x % blocks;
  const uint8_t* const logits = a.logits + row * a.row_stride * kElem;
  uint8_t* const out = a.dlogits + row * a.out_stride * kElem;
  const RowPieces<BF16> p(logits, a.vocab);
  const bool together = ((reinterpret_cast<uintptr_t>(logits) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0;
  int first = part * kGradThreads * kGradPieces + threadIdx.x;
  uint4 r[kGradPieces];
#pragma unroll
  for (int k = 0; k < kGradPieces; ++k) r[k] = p.load(first + k * kGradThreads);
  const int64_t t = a.token_bytes == 4 ? static_cast<const int32_t*>(a.tokens)[row] : static_cast<const int64_t*>(a.tokens)[row];
  const float lse = a.lse[row], g = t >= 0 && t < a.vocab ? a.dlogprob[row] : 0.0f;
  const float h = a.dentropy ? a.dentropy[row] : 0.0f, entropy = a.dentropy ? a.entropy[row] : 0.0f;
  // In powers of two, t = log2 p: dlogits = -p (hs t + ks), plus the token's share.
  const float factor = a.scale * kLog2e;
  float ref = 0.0f, c = lse * kLog2e;
  // Far from zero a float32 lse says little about the sum next to the maximum
  // (at 1024 its step is 2^-13; a row of the type's lowest value would be all
  // certain), and an infinite one nothing (the largest logit times the scale may
  // leave float32): such a row is summed again.
  const bool far = fabsf(lse) > 1024.0f;
  bool dead = false;  // a row of nothing but -inf: every p is 0
  if (far) {
    __shared__ float red[2][kGradThreads / kWave];
    float top = -INFINITY, sum = 0.0f;
    for (int i = threadIdx.x; i < p.pieces(); i += kGradThreads) {
      float v[V];
      unpack_piece<BF16>(p.inside(i, p.load(i)), v);
#pragma unroll
      for (int j = 0; j < V; ++j) top = fmaxf(top, v[j]);
    }
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
    ref = over_waves<kGradThreads / kWave>(top, red[0], [](float x, float y) { return fmaxf(x, y); });
    dead = ref == -INFINITY;
    if (dead) ref = 0.0f;
    for (int i = threadIdx.x; i < p.pieces(); i += kGradThreads) {
      float v[V];
      unpack_piece<BF16>(p.inside(i, p.load(i)), v);
#pragma unroll
      for (int j = 0; j < V; ++j) sum += __builtin_amdgcn_exp2f((v[j] - ref) * factor);
    }
    c = __builtin_log2f(over_waves<kGradThreads / kWave>(wave_sum(sum), red[1], [](float x, float y) { return x + y; }));
    if (dead) c = 0.0f;
    __syncthreads();  // in place: every wave has read the row before one writes
  }
  const float hs = h * a.scale * kLn2, ks = lse != lse ? lse : dead ? 0.0f : __builtin_fmaf(h, entropy, g) * a.scale;
  const float hit = dead ? 0.0f : g * a.scale;
  for (;;) {
#pragma unroll
    for (int k = 0; k < kGradPieces; ++k) {
      const int piece = first + k * kGradThreads;
      const int e = p.index(piece);
      if (e >= p.vocab) break;
      float v[V];
      unpack_piece<BF16>(r[k], v);
      if (far) {
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] -= ref;
      }
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float x = at_least(__builtin_fmaf(v[j], factor, -c), kNothing);
        v[j] = -__builtin_amdgcn_exp2f(x) * __builtin_fmaf(hs, x, ks);
      }
      if (t >= e && t < e + V) {
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] += e + j == t ? hit : 0.0f;
      }
      if (together && e >= 0 && e + V <= p.vocab) {
        *reinterpret_cast<uint4*>(out + static_cast<int64_t>(e) * kElem) = pack_piece<BF16>(v);
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
          if (static_cast<uint32_t>(e + j) < static_cast<uint32_t>(p.vocab)) store_elem<BF16>(out, e + j, v[j]);
      }
    }
    part += blocks;
    if (part >= parts) return;
    first = part * kGradThreads * kGradPieces + threadIdx.x;
#pragma unroll
    for (int k = 0; k < kGradPieces; ++k) r[k] = p.load(first + k * kGradThreads);
  }
}

// Pieces of 16 bytes that a row may span, wherever it starts.
int64_t row_pieces(int64_t vocab, bool bf16) {
  const int64_t v = bf16 ? 8 : 4;
  return (vocab + 2 * v - 2) / v;
}
int grad_parts(int64_t vocab, bool bf16) {
  const int64_t each = kGradThreads * kGradPieces;
  return static_cast<int>((row_pieces(vocab, bf16) + each - 1) / each);
}

template <bool BF16>
hipError_t launch_for(const LogprobArgs& a, hipStream_t s) {
  const int64_t np = row_pieces(a.vocab, BF16);
  const dim3 grid(static_cast<uint32_t>(a.rows));
  if (np <= 256 * 4)
    logprobs_kernel<BF16, 256, 4><<<grid, dim3(256), 0, s>>>(a);
  else if (np <= 1024 * 4)
    logprobs_kernel<BF16, 1024, 4><<<grid, dim3(1024), 0, s>>>(a);
  else if (np <= 1024 * 8)
    logprobs_kernel<BF16, 1024, 8><<<grid, dim3(1024), 0, s>>>(a);
  else if (np <= 1024 * 16)
    logprobs_kernel<BF16, 1024, 16><<<grid, dim3(1024), 0, s>>>(a);
  else
    logprobs_kernel<BF16, 1024, 0><<<grid, dim3(1024), 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

// Blocks of 256 threads, or as many threads, that a call launches.
int64_t logprobs_blocks(int64_t rows, int64_t vocab, bool bf16) { return rows * (row_pieces(vocab, bf16) <= 256 * 4 ? 1 : 4); }

hipError_t launch_logprobs(const LogprobArgs& a, bool bf16, hipStream_t s) {
  return bf16 ? launch_for<true>(a, s) : launch_for<false>(a, s);
}

int64_t logprobs_grad_blocks(int64_t rows, int64_t vocab, bool bf16) { return rows * grad_parts(vocab, bf16); }

hipError_t launch_logprobs_grad(const LogprobArgs& a, bool bf16, hipStream_t s) {
  // In place one block takes the row: it may have to read all of it before it writes.
  const int parts = grad_parts(a.vocab, bf16), blocks = a.dlogits == a.logits ? 1 : parts;
  const dim3 grid(static_cast<uint32_t>(a.rows * blocks)), block(kGradThreads);
  if (bf16)
    logprobs_grad_kernel<true><<<grid, block, 0, s>>>(a, parts, blocks);
  else
    logprobs_grad_kernel<false><<<grid, block, 0, s>>>(a, parts, blocks);
  return hipGetLastError();
}

}  // namespace cq
