// Norm of queries and keys for each head with the position rotation in the
// same pass, out of a projection's output and into a cache, and its gradient.
//
// Per token and head, x of D values with r = rsqrt(mean(x^2) + eps):
// y = x r w (or y = x), then each pair (y_a, y_b) of the first R values turns
// by the angle t = position * freq of the pair:
//   out_a = y_a cos t - y_b sin t,   out_b = y_b cos t + y_a sin t.
// Values v only move.  The gradient turns back by -t, u_a = g_a cos t + g_b sin t,
// u_b = g_b cos t - g_a sin t, and goes through the norm: with z = w u,
//   dx = r (z - x r (r mean(z x))),   dw = sum over tokens and heads of u x r.
//
// Memory bounds it at many tokens: every value is read and written once, 16
// bytes per lane.  8192 bf16 tokens of 32 + 8 heads of 128, with 8 heads of values
// into a cache: 37.5 us for 201 MB, 5.4 TB/s, past a large copy's 4.8 (part stays
// in the last cache), the vector units busy 77%; the gradient 46.3 us for 252 MB,
// 5.4 TB/s, and 7.4 to add the blocks' shares of the weights' gradients.  A head is a team of lanes of 8 values each; a lane needs
// its pairs' other halves too, which lie in the same row, R / 2 values away:
// it loads them as well (from the cache), which costs no exchange between
// lanes.  Angles far out lose their bits in float32 (at position 10^5 the
// angle's step is 2^-8), so the product is taken in float64 and reduced to a
// turn there; sine and cosine are formed once per token, pair and block and
// shared by all heads.
#include "lanes.h"

namespace cq {
namespace {

constexpr int kThreads = 256;
constexpr int kTable = 2048;  // sines and cosines of a block's tokens: 16 KiB
constexpr int kPiece = 8;     // values of a lane

enum Pairing { kNeighbours, kHalves, kHalvesOdd };  // 2i and 2i+1; i and i + R/2, R/2 whole pieces of 8 or not

__device__ __forceinline__ int64_t index_at(const void* p, int bytes, int64_t i) {
  return bytes == 4 ? static_cast<const int32_t*>(p)[i] : static_cast<const int64_t*>(p)[i];
}

// 8 values as loaded.  Addresses looked up in shared memory are global ones,
// which the compiler has to be told: it would take loads that might also meet
// shared memory, and wait for both.
typedef uint32_t u32_x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(1))) u32_x4* global_ptr;
template <bool BF16>
struct Raw8 {
  uint4 r[BF16 ? 1 : 2];
  __device__ __forceinline__ void load(const uint8_t* p) {
#pragma unroll
    for (int i = 0; i < (BF16 ? 1 : 2); ++i) r[i] = __builtin_bit_cast(uint4, static_cast<u32_x4>(((global_ptr)(uint8_t*)p)[i]));
  }
  __device__ __forceinline__ void unpack(float (&v)[8]) const {
    unpack_piece<BF16>(r[0], v);
    if constexpr (!BF16) unpack_piece<BF16>(r[1], v + 4);
  }
  __device__ __forceinline__ void pack(const float (&v)[8]) {
    r[0] = pack_piece<BF16>(v);
    if constexpr (!BF16) r[1] = pack_piece<BF16>(v + 4);
  }
  __device__ __forceinline__ void store(uint8_t* p) const {
#pragma unroll
    for (int i = 0; i < (BF16 ? 1 : 2); ++i) ((global_ptr)p)[i] = __builtin_bit_cast(u32_x4, r[i]);
  }
  __device__ __forceinline__ void choose(bool c, const Raw8& o) {
#pragma unroll
    for (int i = 0; i < (BF16 ? 1 : 2); ++i) r[i] = make_uint4(c ? o.r[i].x : r[i].x, c ? o.r[i].y : r[i].y, c ? o.r[i].z : r[i].z, c ? o.r[i].w : r[i].w);
  }
};

// A team's sum over its L lanes, the same in all of them.
template <int L>
__device__ __forceinline__ float team_sum(float v) {
  v += dpp_move<0xB1>(v);
  v += dpp_move<0x4E>(v);
  if constexpr (L > 4) v += dpp_move<0x141>(v);
  if constexpr (L > 8) v += dpp_move<0x128>(v);
  if constexpr (L > 16) {
    const uint32_t u = __builtin_bit_cast(uint32_t, v);
    const auto ab = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    const uint32_t a = ab[0], b = ab[1];
    v = __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b);
  }
  return v;
}

// Weights of values 8 part .. + 7 in shared memory: quads 0 of all parts, then
// quads 1, so that neighbouring lanes' reads lie side by side in the banks.
constexpr int kMostDim = 256;
__device__ __forceinline__ void load8_weights(const float* w, int part, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(w)[part], b = reinterpret_cast<const float4*>(w)[kMostDim / 8 + part];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ int weight_at(int d) { return (d & 4) * (kMostDim / 8) + (d >> 3) * 4 + (d & 3); }

// What a lane does with its 8 values d0 .. d0 + 7 of every head, without a
// branch: lanes past the head work on its first values and store nothing,
// values that do not turn take cosine 1 and sine 0.
template <bool BF16, int PAIRS>
struct LanePart {
  int d0, half;
  bool live, turns;
  int other;            // kHalves: where its pairs' other halves start
  uint32_t keep, flip;  // kHalves: applied to the other halves' words: cleared if nothing turns; the sign of their sine
  const float2* idle;   // kHalves, nothing turns: instead of the token's cosines and sines
  int entry;            // kHalves: of its first pairs in a token's table
  template <bool BACK>
  __device__ __forceinline__ void place(int part, int head_dim, int rotary, const float2* identity) {
    live = part * kPiece < head_dim;
    d0 = live ? part * kPiece : 0;
    half = rotary / 2;
    turns = d0 < rotary;
    const bool first = d0 < half;
    other = !turns ? d0 : first ? d0 + half : d0 - half;
    keep = turns ? 0xFFFFFFFFu : 0u;
    flip = turns && first != BACK ? (BF16 ? 0x80008000u : 0x80000000u) : 0u;
    idle = turns ? nullptr : identity;
    entry = turns ? (first ? d0 : d0 - half) / 8 : 0;
  }
  // Value j: the place of its pair's other value, or its own if it does not turn.
  __device__ __forceinline__ int partner(int j) const {
    const int d = d0 + j;
    return d < half ? d + half : d < 2 * half ? d - half : d;
  }
  // The pairs' other halves of a row.
  __device__ __forceinline__ void load_others(const uint8_t* row, Raw8<BF16>& o) const {
    if constexpr (PAIRS == kHalves) {
      o.load(row + other * (BF16 ? 2 : 4));
    } else if constexpr (PAIRS == kHalvesOdd) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = load_elem<BF16>(row, partner(j));
      o.r[0] = pack_piece<BF16>(v);
      if constexpr (!BF16) o.r[1] = pack_piece<BF16>(v + 4);
    }
  }
  __device__ __forceinline__ void unpack_others(Raw8<BF16> o, float (&v)[8]) const {
    if constexpr (PAIRS == kHalves) {
#pragma unroll
      for (int i = 0; i < (BF16 ? 1 : 2); ++i) {
        o.r[i].x = (o.r[i].x & keep) ^ flip, o.r[i].y = (o.r[i].y & keep) ^ flip;
        o.r[i].z = (o.r[i].z & keep) ^ flip, o.r[i].w = (o.r[i].w & keep) ^ flip;
      }
    }
    if constexpr (PAIRS != kNeighbours) o.unpack(v);
  }
  // The weights of the pairs' other halves.
  __device__ __forceinline__ void other_weights(const float* w, float (&o)[8]) const {
    if constexpr (PAIRS == kHalves) {
      load8_weights(w, other / 8, o);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = w[weight_at(partner(j))];
    }
  }
  // Turns y, whose pairs' other halves are o (kHalves: with their sine's sign), by a token's table, or back.
  template <bool BACK>
  __device__ __forceinline__ void turn(float (&y)[8], const float (&o)[8], const float2* table) const {
    if constexpr (PAIRS == kNeighbours) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool turns_here = d0 + 2 * i < 2 * half;
        const float2 cs = table[turns_here ? d0 / 2 + i : 0];
        const float s = BACK ? -cs.y : cs.y, a = y[2 * i], b = y[2 * i + 1];
        y[2 * i] = turns_here ? a * cs.x - b * s : a;
        y[2 * i + 1] = turns_here ? b * cs.x + a * s : b;
      }
    } else if constexpr (PAIRS == kHalves) {
      const float4* const from = reinterpret_cast<const float4*>(turns ? table : idle) + entry;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 cs = from[i * (half / 8)];
        y[2 * i] = y[2 * i] * cs.x + o[2 * i] * cs.y;
        y[2 * i + 1] = y[2 * i + 1] * cs.z + o[2 * i + 1] * cs.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int d = d0 + j;
        const bool lower = d < half, turns_here = d < 2 * half;
        const float2 cs = table[lower ? d : turns_here ? d - half : 0];
        const float v = y[j] * cs.x + o[j] * (lower != BACK ? -cs.y : cs.y);
        y[j] = turns_here ? v : y[j];
      }
    }
  }
};

// The (token, head) pairs of a chunk, heads running fastest, dealt to the teams
// in turn; stepped without a division.
struct Place {
  int t, h;
  __device__ __forceinline__ Place(int team, int heads) : t(team / heads), h(team % heads) {}
  __device__ __forceinline__ void step(int tokens_by, int heads_by, int heads) {
    t += tokens_by;
    h += heads_by;
    if (h >= heads) {
      h -= heads;
      ++t;
    }
  }
};

constexpr int kMostTokens = 128;
constexpr int kMostHeads = 256;  // of a block

// Where the heads lie: looked up, since which tensor a head belongs to, times
// two strides, costs more instructions per head than its norm.
struct HeadAt {
  uint64_t in, out;
  uint32_t in_row, out_row;  // bytes from a token to the next
};
__device__ __forceinline__ uint64_t address(const HeadRows& t, int h, int elem) {
  return reinterpret_cast<uint64_t>(t.data) + static_cast<uint64_t>(h) * t.head * elem;
}
__device__ __forceinline__ uint8_t* row_of(uint64_t at, uint32_t row_bytes, uint32_t row) {
  return reinterpret_cast<uint8_t*>(static_cast<uint64_t>(row) * row_bytes + at);
}
// Heads first .. first + count - 1 of the tensors f(head, &in, &out, &its number there).
template <class F>
__device__ __forceinline__ void fill_heads(int first, int count, int elem, HeadAt* to, F f) {
  for (int i = threadIdx.x; i < count; i += kThreads) {
    const HeadRows *in, *out;
    int h;
    f(first + i, &in, &out, &h);
    const HeadAt at{address(*in, h, elem), address(*out, h, elem), static_cast<uint32_t>(in->row * elem), static_cast<uint32_t>(out->row * elem)};
    to[i] = at;
    wait_lds_writes();
    hold_value(at.in);
    hold_value(at.out);
    hold_value(at.in_row);
    hold_value(at.out_row);
  }
}

// Both weights into shared memory, ones where there are none.
__device__ __forceinline__ void fill_weights(const RotateArgs& a, float (&w)[2][kMostDim]) {
  for (int i = threadIdx.x; i < 2 * kMostDim; i += kThreads) {
    const void* const from = i < kMostDim ? a.q_weight : a.k_weight;
    const int d = i % kMostDim;
    float v = 1.0f;
    if (from && d < a.head_dim) v = a.w_bf16 ? bf16_low(static_cast<const uint16_t*>(from)[d]) : static_cast<const float*>(from)[d];
    w[i / kMostDim][weight_at(d)] = v;
    wait_lds_writes();
    hold_value(v);
  }
}

// Cosines and sines of tokens first .. first + count - 1 into shared memory:
// per token in order of the pairs, or (kHalves) pairs 0 and 1 of all runs of 8
// pairs, then pairs 2 and 3, and so on.
template <int PAIRS>
__device__ __forceinline__ void fill_table(const RotateArgs& a, int64_t first, int count, float2* table) {
  const int half = a.rotary_dim / 2;
  for (int i = threadIdx.x; i < count * half; i += kThreads) {
    const int t = i / half, j = i % half;
    const double turns = static_cast<double>(index_at(a.positions, a.position_bytes, first + t)) *
                         (static_cast<double>(a.freqs[j]) * 0.3183098861837906715);  // half turns
    // Reduced to a turn, the angle in two floats: sin(h + l) = sin h + l cos h.
    const double part = turns - 2.0 * rint(0.5 * turns);
    const float high = static_cast<float>(part), low = static_cast<float>(part - high) * 3.14159265f;
    float s, c;
    sincospif(high, &s, &c);
    const float2 cs = make_float2(__builtin_fmaf(-low, s, c), __builtin_fmaf(low, c, s));
    const int at = PAIRS == kHalves ? (j & 6) * (half / 8) + (j >> 3) * 2 + (j & 1) : j;
    table[t * half + at] = cs;
    wait_lds_writes();
    hold_value(cs.x);
    hold_value(cs.y);
  }
  __syncthreads();
}
__device__ __forceinline__ void fill_identity(float2* identity) {
  if (threadIdx.x < kMostDim / 2) {
    const float2 cs = make_float2(1.0f, 0.0f);
    identity[threadIdx.x] = cs;
    wait_lds_writes();
    hold_value(cs.x);
    hold_value(cs.y);
  }
}

// Blocks walk over chunks of `tokens` tokens (a launch per block and chunk
// would spend its time on weights and first loads: 8192 bf16 tokens of 48 heads
// of 128, one token per block 151 us) and take of each the heads (queries',
// keys', values') blockIdx.y * heads .. + heads - 1.  A team has its next two
// heads' loads under way while it computes one: three sets of registers in
// turn (a set moved on to the next would wait for its loads), and no branch
// between a load and its use, so that the waits count exactly.
template <bool BF16, int L, int PAIRS>
__global__ void __launch_bounds__(kThreads, PAIRS == kHalvesOdd ? 3 : 4) rotate_kernel(RotateArgs a, int tokens, int heads, int64_t chunks) {
  constexpr int kElem = BF16 ? 2 : 4, kTeams = kThreads / L;
  __shared__ __attribute__((aligned(16))) float2 table[kTable];
  __shared__ __attribute__((aligned(16))) float2 identity[kMostDim / 2];
  __shared__ __attribute__((aligned(16))) float weights[2][kMostDim];
  __shared__ __attribute__((aligned(16))) HeadAt head_at[kMostHeads];
  __shared__ int rows[kMostTokens];
  LanePart<BF16, PAIRS> lane;
  lane.template place<false>(threadIdx.x % L, a.head_dim, a.rotary_dim, identity);
  const int total = a.q_heads + a.kv_heads * (a.v.data ? 2 : 1), rotated = a.q_heads + a.kv_heads;
  const int h0 = blockIdx.y * heads, nh = total - h0 < heads ? total - h0 : heads, half = a.rotary_dim / 2;
  fill_heads(h0, nh, kElem, head_at, [&](int h, const HeadRows** in, const HeadRows** out, int* number) __attribute__((always_inline)) {
    const bool is_q = h < a.q_heads, is_v = h >= rotated;
    *in = is_q ? &a.q : is_v ? &a.v : &a.k;
    *out = is_q ? &a.q_out : is_v ? &a.v_out : &a.k_out;
    *number = h - (is_q ? 0 : is_v ? rotated : a.q_heads);
  });
  __syncthreads();

  struct Item {
    Raw8<BF16> y, o;
  };
  const Place first(threadIdx.x / L, nh);
  const int tokens_by = kTeams / nh, heads_by = kTeams % nh;
  const float per_value = 1.0f / static_cast<float>(a.head_dim);
  for (int64_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const uint32_t t0 = static_cast<uint32_t>(c * tokens);
    const int nt = a.n - t0 < tokens ? static_cast<int>(a.n - t0) : tokens, turns = (nt * nh + kTeams - 1) / kTeams;
    Place at = first, ahead = first;
    // The heads past a chunk's last read its last token once more.
    auto load = [&](Item& it) __attribute__((always_inline)) {
      const HeadAt& from = head_at[ahead.h];
      const uint8_t* const row = row_of(from.in, from.in_row, t0 + (ahead.t < nt ? ahead.t : nt - 1));
      it.y.load(row + lane.d0 * kElem);
      lane.load_others(row, it.o);
      ahead.step(tokens_by, heads_by, nh);
    };
    Item i0, i1, i2;
    load(i0);
    load(i1);
    if (c == blockIdx.x) {
      fill_weights(a, weights);
      fill_identity(identity);
    } else {
      __syncthreads();  // the last chunk's table is read
    }
    if (a.slots)
      for (int i = threadIdx.x; i < nt; i += kThreads) {
        const int64_t slot = index_at(a.slots, a.slot_bytes, t0 + i);
        const int row = slot >= 0 && slot < a.cache_rows ? static_cast<int>(slot) : -1;
        rows[i] = row;  // of the cache, below 0: none
        wait_lds_writes();
        hold_value(row);
      }
    fill_table<PAIRS>(a, t0, nt, table);
    auto work = [&](const Item& it) __attribute__((always_inline)) {
      const HeadAt& to = head_at[at.h];
      const int t = at.t < nt ? at.t : nt - 1, h = h0 + at.h;
      const bool is_q = h < a.q_heads, is_v = h >= rotated;
      float y[8], o[8], v[8], r = 1.0f;
      it.y.unpack(y);
      lane.unpack_others(it.o, o);
      if (a.norm) {
        float ss = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = __builtin_fmaf(y[j], y[j], ss);
        r = rsqrtf(__builtin_fmaf(team_sum<L>(lane.live ? ss : 0.0f), per_value, a.eps));
      }
      const float* const w = weights[is_q ? 0 : 1];
      load8_weights(w, lane.d0 / 8, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] *= r * v[j];
      if constexpr (PAIRS != kNeighbours) {
        lane.other_weights(w, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] *= r * v[j];
      }
      lane.template turn<false>(y, o, table + t * half);
      int row = static_cast<int>(t0 + t);
      if (a.slots && !is_q) row = rows[t];
      Raw8<BF16> out;
      out.pack(y);
      out.choose(is_v, it.y);
      if (lane.live && at.t < nt && row >= 0) out.store(row_of(to.out, to.out_row, row) + lane.d0 * kElem);
      at.step(tokens_by, heads_by, nh);
    };
    for (int i = 0;;) {
      load(i2);
      work(i0);
      if (++i >= turns) break;
      load(i0);
      work(i1);
      if (++i >= turns) break;
      load(i1);
      work(i2);
      if (++i >= turns) break;
    }
  }
}

// The gradient's blocks walk over chunks of tokens; the shares of the weights'
// gradients stay in registers until the last one.
template <bool BF16, int L, int PAIRS>
__global__ void __launch_bounds__(kThreads, BF16 && PAIRS != kHalvesOdd ? 4 : 3) rotate_grad_kernel(RotateArgs a, int tokens, int heads, int64_t chunks) {
  constexpr int kElem = BF16 ? 2 : 4, kTeams = kThreads / L;
  __shared__ __attribute__((aligned(16))) float2 table[kTable];
  __shared__ __attribute__((aligned(16))) float2 identity[kMostDim / 2];
  __shared__ __attribute__((aligned(16))) float weights[2][kMostDim];
  __shared__ __attribute__((aligned(16))) HeadAt grad_at[kMostHeads], x_at[kMostHeads];
  LanePart<BF16, PAIRS> lane;
  lane.template place<true>(threadIdx.x % L, a.head_dim, a.rotary_dim, identity);
  const int total = a.q_heads + a.kv_heads, half = a.rotary_dim / 2;
  const int h0 = blockIdx.y * heads, nh = total - h0 < heads ? total - h0 : heads;
  float dqw[8], dkw[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) dqw[j] = dkw[j] = 0.0f;
  auto of_head = [&](const HeadRows& q_in, const HeadRows& k_in) __attribute__((always_inline)) {
    return [&a, &q_in, &k_in](int h, const HeadRows** in, const HeadRows** out, int* number) __attribute__((always_inline)) {
      const bool is_q = h < a.q_heads;
      *in = is_q ? &q_in : &k_in;
      *out = is_q ? &a.q_out : &a.k_out;
      *number = h - (is_q ? 0 : a.q_heads);
    };
  };
  fill_heads(h0, nh, kElem, grad_at, of_head(a.dq, a.dk));
  if (a.norm) fill_heads(h0, nh, kElem, x_at, of_head(a.q, a.k));
  __syncthreads();

  struct Item {
    Raw8<BF16> u, o, x;
  };
  const Place first(threadIdx.x / L, nh);
  const int tokens_by = kTeams / nh, heads_by = kTeams % nh;
  const float per_value = 1.0f / static_cast<float>(a.head_dim);
  for (int64_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const uint32_t t0 = static_cast<uint32_t>(c * tokens);
    const int nt = a.n - t0 < tokens ? static_cast<int>(a.n - t0) : tokens, turns = (nt * nh + kTeams - 1) / kTeams;
    Place at = first, ahead = first;
    auto load = [&](Item& it) __attribute__((always_inline)) {
      const uint32_t token = t0 + (ahead.t < nt ? ahead.t : nt - 1);
      const HeadAt& from = grad_at[ahead.h];
      const uint8_t* const row = row_of(from.in, from.in_row, token);
      it.u.load(row + lane.d0 * kElem);
      lane.load_others(row, it.o);
      if (a.norm) it.x.load(row_of(x_at[ahead.h].in, x_at[ahead.h].in_row, token) + lane.d0 * kElem);
      ahead.step(tokens_by, heads_by, nh);
    };
    Item i0, i1, i2;
    load(i0);
    load(i1);
    if (c == blockIdx.x) {
      fill_weights(a, weights);
      fill_identity(identity);
    } else {
      __syncthreads();  // the last chunk's table is read
    }
    fill_table<PAIRS>(a, t0, nt, table);
    auto work = [&](const Item& it) __attribute__((always_inline)) {
      const HeadAt& to = grad_at[at.h];
      const int t = at.t < nt ? at.t : nt - 1;
      const bool is_q = h0 + at.h < a.q_heads, exists = at.t < nt;
      float u[8], o[8];
      it.u.unpack(u);
      lane.unpack_others(it.o, o);
      lane.template turn<true>(u, o, table + t * half);
      if (a.norm) {
        float x[8], w[8], ss = 0.0f, dot = 0.0f;
        it.x.unpack(x);
        load8_weights(weights[is_q ? 0 : 1], lane.d0 / 8, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          ss = __builtin_fmaf(x[j], x[j], ss);
          dot = __builtin_fmaf(u[j] * w[j], x[j], dot);
        }
        const float r = rsqrtf(__builtin_fmaf(team_sum<L>(lane.live ? ss : 0.0f), per_value, a.eps));
        const float k = r * (team_sum<L>(lane.live ? dot : 0.0f) * per_value);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] *= r;
        if (exists && is_q) {
#pragma unroll
          for (int j = 0; j < 8; ++j) dqw[j] = __builtin_fmaf(u[j], x[j], dqw[j]);
        }
        if (exists && !is_q) {
#pragma unroll
          for (int j = 0; j < 8; ++j) dkw[j] = __builtin_fmaf(u[j], x[j], dkw[j]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) u[j] = r * __builtin_fmaf(-x[j], k, u[j] * w[j]);
      }
      Raw8<BF16> out;
      out.pack(u);
      if (lane.live && exists) out.store(row_of(to.out, to.out_row, t0 + t) + lane.d0 * kElem);
      at.step(tokens_by, heads_by, nh);
    };
    for (int i = 0;;) {
      load(i2);
      work(i0);
      if (++i >= turns) break;
      load(i0);
      work(i1);
      if (++i >= turns) break;
      load(i1);
      work(i2);
      if (++i >= turns) break;
    }
  }
  if (!a.part) return;
  // The teams' shares in team order.
  float* const share = reinterpret_cast<float*>(table);  // [teams][L * 8], 2048 floats
  const int64_t block = static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
    uint4 w[2];
    w[0] = pack_piece<false>(which ? dkw : dqw);
    w[1] = pack_piece<false>((which ? dkw : dqw) + 4);
    reinterpret_cast<uint4*>(share)[2 * threadIdx.x] = w[0];
    reinterpret_cast<uint4*>(share)[2 * threadIdx.x + 1] = w[1];
    hold_until_lds_written(w);
    __syncthreads();
    for (int d = threadIdx.x; d < a.head_dim; d += kThreads) {
      float sum = 0.0f;
      for (int t = 0; t < kTeams; ++t) sum += share[t * L * kPiece + d];
      a.part[(block * 2 + which) * a.head_dim + d] = sum;
    }
  }
}

// The blocks' shares in block order, 16 runs of blocks side by side.
// Latency: 7.4 us for 1024 blocks of 128 values (with 32 loads in flight 7.5).
constexpr int kRuns = 16;
__global__ void __launch_bounds__(kRuns* kWave) rotate_weight_kernel(const float* part, int blocks, int head_dim, float* dq, float* dk) {
  __shared__ float run[kRuns][kWave];
  const int lane = threadIdx.x % kWave, r = threadIdx.x / kWave;
  const int d = blockIdx.x * kWave + lane, which = blockIdx.y;
  const int each = (blocks + kRuns - 1) / kRuns, end = (r + 1) * each < blocks ? (r + 1) * each : blocks;
  float sum = 0.0f;
  for (int b = r * each; b < end; b += 16) {
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = d < head_dim && b + i < end ? part[(static_cast<int64_t>(b + i) * 2 + which) * head_dim + d] : 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) sum += v[i];
  }
  run[r][lane] = sum;
  wait_lds_writes();
  hold_value(sum);
  __syncthreads();
  float* const out = which ? dk : dq;
  if (r || d >= head_dim || !out) return;
#pragma unroll
  for (int i = 1; i < kRuns; ++i) sum += run[i][lane];
  out[d] = sum;
}

int lanes_of(int head_dim) { return head_dim <= 32 ? 4 : head_dim <= 64 ? 8 : head_dim <= 128 ? 16 : 32; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Tokens of a chunk: enough for each team to take four heads and for each
// thread to form a sine, fewer while that leaves compute units idle (1000 float32
// tokens, 8 + 2 heads of 64: 5.2 us and gradient 6.4 + 3.7 in 334 blocks, 5.8 and
// 10.2 + 7.2 in 1000).
int tokens_of(int64_t n, int heads, int head_dim) {
  const int teams = kThreads / lanes_of(head_dim);
  const int64_t most = 4 * teams / heads < 4 ? 4 : 4 * teams / heads, fill = n / kCus;
  const int64_t tokens = fill < most ? fill : most;
  return static_cast<int>(tokens < 1 ? 1 : tokens);
}
// Heads of a block: all, or one token's heads over several blocks while there
// are few tokens.
int heads_of(int64_t n, int total, int tokens, int head_dim) {
  const int teams = kThreads / lanes_of(head_dim), heads = tokens == 1 && n * ceil_div(total, teams) <= 8 * kCus ? teams : total;
  return heads < kMostHeads ? heads : kMostHeads;
}
constexpr int kMostBlocks = 4 * kCus;  // as many as fit the card at once

template <bool BF16, int L, int PAIRS>
hipError_t launch_at(const RotateArgs& a, hipStream_t s) {
  const int total = a.q_heads + a.kv_heads * (a.v.data ? 2 : 1);
  const int tokens = tokens_of(a.n, total, a.head_dim);
  const int heads = heads_of(a.n, total, tokens, a.head_dim);
  const int64_t chunks = ceil_div(a.n, tokens);
  rotate_kernel<BF16, L, PAIRS><<<dim3(static_cast<uint32_t>(chunks < kMostBlocks ? chunks : kMostBlocks),
                                       static_cast<uint32_t>(ceil_div(total, heads))),
                                  dim3(kThreads), 0, s>>>(a, tokens, heads, chunks);
  return hipGetLastError();
}
template <bool BF16, int L, int PAIRS>
hipError_t launch_grad_at(const RotateArgs& a, int blocks, hipStream_t s) {
  const int total = a.q_heads + a.kv_heads, tokens = tokens_of(a.n, total, a.head_dim), parts = static_cast<int>(ceil_div(total, kMostHeads));
  rotate_grad_kernel<BF16, L, PAIRS><<<dim3(blocks / parts, parts), dim3(kThreads), 0, s>>>(
      a, tokens, total < kMostHeads ? total : kMostHeads, ceil_div(a.n, tokens));
  return hipGetLastError();
}

int pairing(const RotateArgs& a) {
  return a.interleaved || a.rotary_dim == 0 ? kNeighbours : a.rotary_dim % 16 == 0 ? kHalves : kHalvesOdd;
}

// Calls f(BF16, lanes, pairing) with compile-time values.
template <bool BF16, int L, class F>
hipError_t by_pairing(const RotateArgs& a, F f) {
  switch (pairing(a)) {
    case kNeighbours: return f(std::integral_constant<int, L>{}, std::integral_constant<int, kNeighbours>{});
    case kHalves: return f(std::integral_constant<int, L>{}, std::integral_constant<int, kHalves>{});
    default: return f(std::integral_constant<int, L>{}, std::integral_constant<int, kHalvesOdd>{});
  }
}
template <bool BF16, class F>
hipError_t by_shape(const RotateArgs& a, F f) {
  switch (lanes_of(a.head_dim)) {
    case 4: return by_pairing<BF16, 4>(a, f);
    case 8: return by_pairing<BF16, 8>(a, f);
    case 16: return by_pairing<BF16, 16>(a, f);
    default: return by_pairing<BF16, 32>(a, f);
  }
}
template <bool BF16>
hipError_t forward(const RotateArgs& a, hipStream_t s) {
  return by_shape<BF16>(a, [&](auto l, auto p) { return launch_at<BF16, decltype(l)::value, decltype(p)::value>(a, s); });
}
template <bool BF16>
hipError_t backward(const RotateArgs& a, int blocks, hipStream_t s) {
  return by_shape<BF16>(a, [&](auto l, auto p) { return launch_grad_at<BF16, decltype(l)::value, decltype(p)::value>(a, blocks, s); });
}

}  // namespace

hipError_t launch_rotate_heads(const RotateArgs& a, bool bf16, hipStream_t s) {
  return bf16 ? forward<true>(a, s) : forward<false>(a, s);
}

// One chunk of tokens per block, up to 4 blocks per CU, for each kMostHeads heads.
int rotate_grad_blocks(int64_t n, int q_heads, int kv_heads, int head_dim) {
  const int total = q_heads + kv_heads;
  const int64_t chunks = ceil_div(n, tokens_of(n, total, head_dim));
  return static_cast<int>((chunks < kMostBlocks ? chunks : kMostBlocks) * ceil_div(total, kMostHeads));
}

hipError_t launch_rotate_heads_grad(RotateArgs a, bool bf16, float* dq_weight, float* dk_weight, float* ws, hipStream_t s) {
  const int blocks = rotate_grad_blocks(a.n, a.q_heads, a.kv_heads, a.head_dim);
  const bool weights = dq_weight || dk_weight;
  a.part = weights ? ws : nullptr;
  const hipError_t e = bf16 ? backward<true>(a, blocks, s) : backward<false>(a, blocks, s);
  if (e != hipSuccess || !weights) return e;
  rotate_weight_kernel<<<dim3(static_cast<uint32_t>(ceil_div(a.head_dim, kWave)), 2), dim3(kRuns * kWave), 0, s>>>(
      ws, blocks, a.head_dim, dq_weight, dk_weight);
  return hipGetLastError();
}

}  // namespace cq
