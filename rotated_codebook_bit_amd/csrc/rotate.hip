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
// bytes per lane.  A head is a team of lanes of 8 values each; a lane needs
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

// 8 values as loaded.
template <bool BF16>
struct Raw8 {
  uint4 r[BF16 ? 1 : 2];
  __device__ __forceinline__ void load(const uint8_t* p) {
#pragma unroll
    for (int i = 0; i < (BF16 ? 1 : 2); ++i) r[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void unpack(float (&v)[8]) const {
    unpack_piece<BF16>(r[0], v);
    if constexpr (!BF16) unpack_piece<BF16>(r[1], v + 4);
  }
};
template <bool BF16>
__device__ __forceinline__ void store8(uint8_t* p, const float (&v)[8]) {
  if constexpr (BF16) {
    *reinterpret_cast<uint4*>(p) = pack_piece<true>(v);
  } else {
    reinterpret_cast<uint4*>(p)[0] = pack_piece<false>(v);
    reinterpret_cast<uint4*>(p)[1] = pack_piece<false>(v + 4);
  }
}

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

__device__ __forceinline__ void load8_shared(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

// What a lane does with its 8 values d0 .. d0 + 7 of every head.
template <int PAIRS>
struct LanePart {
  int d0, half;
  bool live, turns, first;  // inside the head; some values turn; kHalves: all are first of their pair
  int other;                // kHalves: where its pairs' other halves start
  __device__ __forceinline__ LanePart(int part, int head_dim, int rotary) {
    d0 = part * kPiece;
    half = rotary / 2;
    live = d0 < head_dim;
    turns = live && d0 < rotary;
    first = d0 < half;
    other = first ? d0 + half : d0 - half;
  }
  // Value j: the place of its pair's other value, or its own if it does not turn.
  __device__ __forceinline__ int place(int j) const {
    const int d = d0 + j;
    return d < half ? d + half : d < 2 * half ? d - half : d;
  }
  // The pairs' other halves of a row, as they lie in memory.
  template <bool BF16>
  __device__ __forceinline__ void load_others(const uint8_t* row, Raw8<BF16>& o) const {
    if constexpr (PAIRS == kHalves) {
      o.load(row + other * (BF16 ? 2 : 4));
    } else if constexpr (PAIRS == kHalvesOdd) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = load_elem<BF16>(row, place(j));
      o.r[0] = pack_piece<BF16>(v);
      if constexpr (!BF16) o.r[1] = pack_piece<BF16>(v + 4);
    }
  }
  // The weights of the pairs' other halves.
  __device__ __forceinline__ void other_weights(const float* w, float (&o)[8]) const {
    if constexpr (PAIRS == kHalves) {
      load8_shared(w + other, o);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = w[place(j)];
    }
  }
  // Turns y, whose pairs' other halves are o, by the token's table, or back.
  template <bool BACK>
  __device__ __forceinline__ void turn(float (&y)[8], const float (&o)[8], const float2* table) const {
    if constexpr (PAIRS == kNeighbours) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (d0 + 2 * i >= 2 * half) continue;
        const float2 cs = table[d0 / 2 + i];
        const float s = BACK ? -cs.y : cs.y, a = y[2 * i], b = y[2 * i + 1];
        y[2 * i] = a * cs.x - b * s;
        y[2 * i + 1] = b * cs.x + a * s;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int d = d0 + j;
        if (PAIRS == kHalvesOdd && d >= 2 * half) continue;
        const bool lower = PAIRS == kHalves ? first : d < half;
        const float2 cs = table[lower ? d : d - half];
        y[j] = y[j] * cs.x + o[j] * (lower != BACK ? -cs.y : cs.y);
      }
    }
  }
};

// The tensor that a head belongs to, field by field: a choice between the
// structs themselves would be made between their addresses, and every use then
// load from memory and wait for all loads under way.
__device__ __forceinline__ HeadRows pick(bool first, const HeadRows& a, const HeadRows& b) {
  return HeadRows{first ? a.data : b.data, first ? a.row : b.row, first ? a.head : b.head};
}

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

constexpr int kMostDim = 256, kMostTokens = 128;
// Both weights into shared memory, ones where there are none.
__device__ __forceinline__ void fill_weights(const RotateArgs& a, float (&w)[2][kMostDim]) {
  for (int i = threadIdx.x; i < 2 * kMostDim; i += kThreads) {
    const void* const from = i < kMostDim ? a.q_weight : a.k_weight;
    const int d = i % kMostDim;
    float v = 1.0f;
    if (from && d < a.head_dim) v = a.w_bf16 ? bf16_low(static_cast<const uint16_t*>(from)[d]) : static_cast<const float*>(from)[d];
    w[i / kMostDim][d] = v;
    wait_lds_writes();
    hold_value(v);
  }
}

// Cosines and sines of tokens first .. first + count - 1 into shared memory.
__device__ __forceinline__ void fill_table(const RotateArgs& a, int64_t first, int count, float2* table) {
  const int half = a.rotary_dim / 2;
  for (int i = threadIdx.x; i < count * half; i += kThreads) {
    const double turns = static_cast<double>(index_at(a.positions, a.position_bytes, first + i / half)) *
                         (static_cast<double>(a.freqs[i % half]) * 0.3183098861837906715);  // half turns
    // Reduced to a turn, the angle in two floats: sin(h + l) = sin h + l cos h.
    const double part = turns - 2.0 * rint(0.5 * turns);
    const float high = static_cast<float>(part), low = static_cast<float>(part - high) * 3.14159265f;
    float s, c;
    sincospif(high, &s, &c);
    const float2 cs = make_float2(__builtin_fmaf(-low, s, c), __builtin_fmaf(low, c, s));
    table[i] = cs;
    wait_lds_writes();
    hold_value(cs.x);
    hold_value(cs.y);
  }
  __syncthreads();
}

// Blocks walk over chunks of `tokens` tokens (a launch per block and chunk
// would spend its time on weights and first loads: 8192 bf16 tokens of 48 heads
// of 128, one token per block 151 us) and take of each the heads (queries',
// keys', values') blockIdx.y * heads .. + heads - 1.  A team has its next two
// heads' loads under way while it computes one.
template <bool BF16, int L, int PAIRS>
__global__ void __launch_bounds__(kThreads, 4) rotate_kernel(RotateArgs a, int tokens, int heads, int64_t chunks) {
  constexpr int kElem = BF16 ? 2 : 4, kTeams = kThreads / L;
  __shared__ __attribute__((aligned(16))) float2 table[kTable];
  __shared__ __attribute__((aligned(16))) float weights[2][kMostDim];
  __shared__ int64_t rows[kMostTokens];
  const LanePart<PAIRS> lane(threadIdx.x % L, a.head_dim, a.rotary_dim);
  const int total = a.q_heads + a.kv_heads * (a.v.data ? 2 : 1), rotated = a.q_heads + a.kv_heads;
  const int h0 = blockIdx.y * heads, nh = total - h0 < heads ? total - h0 : heads, half = a.rotary_dim / 2;
  fill_weights(a, weights);

  const HeadRows q_in = a.q, k_in = a.k, v_in = a.v, q_to = a.q_out, k_to = a.k_out, v_to = a.v_out;
  struct Item {
    Raw8<BF16> y, o;
  };
  const Place first(threadIdx.x / L, nh);
  const int tokens_by = kTeams / nh, heads_by = kTeams % nh;
  const float per_value = 1.0f / static_cast<float>(a.head_dim);
  for (int64_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int64_t t0 = c * tokens;
    const int nt = a.n - t0 < tokens ? static_cast<int>(a.n - t0) : tokens;
    auto load = [&](const Place& at, Item& it) __attribute__((always_inline)) {
      const int64_t token = t0 + at.t;
      const int h = h0 + at.h;
      const bool is_q = h < a.q_heads, is_v = h >= rotated;
      const HeadRows from = pick(is_q, q_in, pick(is_v, v_in, k_in));
      const uint8_t* const row = from.data + (token * from.row + (h - (is_q ? 0 : is_v ? rotated : a.q_heads)) * from.head) * kElem;
      if (lane.live) it.y.load(row + lane.d0 * kElem);
      if (lane.turns && !is_v) lane.template load_others<BF16>(row, it.o);
    };
    // Three heads in turn: one computed, two on their way.
    Item now{}, next{}, last{};
    Place at = first, ahead = first;
    if (ahead.t < nt) load(ahead, now);
    ahead.step(tokens_by, heads_by, nh);
    if (ahead.t < nt) load(ahead, next);
    __syncthreads();  // the last chunk's table is read
    if (a.slots)
      for (int i = threadIdx.x; i < nt; i += kThreads) {
        const int64_t slot = index_at(a.slots, a.slot_bytes, t0 + i), row = slot < a.cache_rows ? slot : -1;
        rows[i] = row;  // of the cache, below 0: none
        wait_lds_writes();
        hold_value(row);
      }
    fill_table(a, t0, nt, table);
    while (at.t < nt) {
      ahead.step(tokens_by, heads_by, nh);
      if (ahead.t < nt) load(ahead, last);
      const int h = h0 + at.h;
      const bool is_q = h < a.q_heads, is_v = h >= rotated;
      float y[8], o[8];
      now.y.unpack(y);
      if (!is_v) {
        now.o.unpack(o);
        if (a.norm) {
          float ss = 0.0f;
#pragma unroll
          for (int j = 0; j < 8; ++j) ss = __builtin_fmaf(y[j], y[j], ss);
          const float r = rsqrtf(__builtin_fmaf(team_sum<L>(ss), per_value, a.eps));
          const float* const w = weights[is_q ? 0 : 1];
          float v[8];
          load8_shared(w + (lane.live ? lane.d0 : 0), v);
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] *= r * v[j];
          if (PAIRS != kNeighbours && lane.turns) {
            lane.other_weights(w, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] *= r * v[j];
          }
        }
        if (lane.turns) lane.template turn<false>(y, o, table + at.t * half);
      }
      int64_t row = t0 + at.t;
      if (a.slots && !is_q) row = rows[at.t];
      if (lane.live && row >= 0) {
        const HeadRows to = pick(is_q, q_to, pick(is_v, v_to, k_to));
        store8<BF16>(to.data + (row * to.row + (h - (is_q ? 0 : is_v ? rotated : a.q_heads)) * to.head + lane.d0) * kElem, y);
      }
      now = next;
      next = last;
      at.step(tokens_by, heads_by, nh);
    }
  }
}

// The gradient's blocks walk over chunks of tokens; the shares of the weights'
// gradients stay in registers until the last one.
template <bool BF16, int L, int PAIRS>
__global__ void __launch_bounds__(kThreads, 4) rotate_grad_kernel(RotateArgs a, int tokens, int64_t chunks) {
  constexpr int kElem = BF16 ? 2 : 4, kTeams = kThreads / L;
  __shared__ __attribute__((aligned(16))) float2 table[kTable];
  __shared__ __attribute__((aligned(16))) float weights[2][kMostDim];
  const LanePart<PAIRS> lane(threadIdx.x % L, a.head_dim, a.rotary_dim);
  const int heads = a.q_heads + a.kv_heads, half = a.rotary_dim / 2;
  const HeadRows dq_in = a.dq, dk_in = a.dk, q_in = a.q, k_in = a.k, dq_to = a.q_out, dk_to = a.k_out;
  float dqw[8], dkw[8];
  fill_weights(a, weights);
#pragma unroll
  for (int j = 0; j < 8; ++j) dqw[j] = dkw[j] = 0.0f;

  const Place first(threadIdx.x / L, heads);
  const int tokens_by = kTeams / heads, heads_by = kTeams % heads;
  const float per_value = 1.0f / static_cast<float>(a.head_dim);
  for (int64_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int64_t t0 = c * tokens;
    const int nt = a.n - t0 < tokens ? static_cast<int>(a.n - t0) : tokens;
    struct Item {
      Raw8<BF16> u, o, x;
    };
    auto load = [&](const Place& at, Item& it) __attribute__((always_inline)) {
      const int64_t token = t0 + at.t;
      const bool is_q = at.h < a.q_heads;
      const int64_t h = at.h - (is_q ? 0 : a.q_heads);
      const HeadRows grad = pick(is_q, dq_in, dk_in), from = pick(is_q, q_in, k_in);
      const uint8_t* const g_row = grad.data + (token * grad.row + h * grad.head) * kElem;
      if (lane.live) it.u.load(g_row + lane.d0 * kElem);
      if (lane.turns) lane.template load_others<BF16>(g_row, it.o);
      if (a.norm && lane.live) it.x.load(from.data + (token * from.row + h * from.head + lane.d0) * kElem);
    };
    Item now{}, next{}, last{};
    Place at = first, ahead = first;
    if (ahead.t < nt) load(ahead, now);
    ahead.step(tokens_by, heads_by, heads);
    if (ahead.t < nt) load(ahead, next);
    __syncthreads();  // the last chunk's table is read
    fill_table(a, t0, nt, table);
    while (at.t < nt) {
      ahead.step(tokens_by, heads_by, heads);
      if (ahead.t < nt) load(ahead, last);
      const int64_t token = t0 + at.t;
      const bool is_q = at.h < a.q_heads;
      const int64_t h = at.h - (is_q ? 0 : a.q_heads);
      const HeadRows to = pick(is_q, dq_to, dk_to);
      float u[8], o[8];
      now.u.unpack(u);
      now.o.unpack(o);
      if (lane.turns) lane.template turn<true>(u, o, table + at.t * half);
      if (a.norm) {
        float x[8], w[8], ss = 0.0f, dot = 0.0f;
        now.x.unpack(x);
        load8_shared(weights[is_q ? 0 : 1] + (lane.live ? lane.d0 : 0), w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          ss = __builtin_fmaf(x[j], x[j], ss);
          dot = __builtin_fmaf(u[j] * w[j], x[j], dot);
        }
        const float r = rsqrtf(__builtin_fmaf(team_sum<L>(ss), per_value, a.eps)), k = r * (team_sum<L>(dot) * per_value);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float xr = x[j] * r, g = u[j];
          u[j] = r * __builtin_fmaf(-xr, k, g * w[j]);
          if (is_q)
            dqw[j] = __builtin_fmaf(g, xr, dqw[j]);
          else
            dkw[j] = __builtin_fmaf(g, xr, dkw[j]);
        }
      }
      if (lane.live) store8<BF16>(to.data + (token * to.row + h * to.head + lane.d0) * kElem, u);
      now = next;
      next = last;
      at.step(tokens_by, heads_by, heads);
    }
  }
  if (!a.part) return;
  // The teams' shares in team order.
  float* const share = reinterpret_cast<float*>(table);  // [teams][L * 8], 2048 floats
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
      a.part[(static_cast<int64_t>(blockIdx.x) * 2 + which) * a.head_dim + d] = sum;
    }
  }
}

// The blocks' shares in block order, 16 runs of blocks side by side.
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
// thread to form a sine, fewer while that leaves compute units idle.
int tokens_of(int64_t n, int heads, int head_dim) {
  const int teams = kThreads / lanes_of(head_dim);
  const int64_t most = 4 * teams / heads < 4 ? 4 : 4 * teams / heads, fill = n / (4 * kCus);
  const int64_t tokens = fill < most ? fill : most;
  return static_cast<int>(tokens < 1 ? 1 : tokens);
}
// Heads of a block: all, or one token's heads over several blocks while there
// are few tokens.
int heads_of(int64_t n, int total, int tokens, int head_dim) {
  const int teams = kThreads / lanes_of(head_dim);
  return tokens == 1 && n * ceil_div(total, teams) <= 8 * kCus ? teams : total;
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
  const int tokens = tokens_of(a.n, a.q_heads + a.kv_heads, a.head_dim);
  rotate_grad_kernel<BF16, L, PAIRS><<<dim3(blocks), dim3(kThreads), 0, s>>>(a, tokens, ceil_div(a.n, tokens));
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

// One chunk of tokens per block, up to 4 blocks per CU of the MI355X.
int rotate_grad_blocks(int64_t n, int q_heads, int kv_heads, int head_dim) {
  const int64_t chunks = ceil_div(n, tokens_of(n, q_heads + kv_heads, head_dim));
  return static_cast<int>(chunks < 1024 ? chunks : 1024);
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
