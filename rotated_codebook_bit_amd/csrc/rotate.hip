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

template <bool BF16>
__device__ __forceinline__ void load8(const uint8_t* p, float (&v)[8]) {
  if constexpr (BF16) {
    unpack_piece<true>(*reinterpret_cast<const uint4*>(p), v);
  } else {
    unpack_piece<false>(reinterpret_cast<const uint4*>(p)[0], v);
    unpack_piece<false>(reinterpret_cast<const uint4*>(p)[1], v + 4);
  }
}
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
  // The pairs' other halves of a row.
  template <bool BF16>
  __device__ __forceinline__ void load_others(const uint8_t* row, float (&o)[8]) const {
    if constexpr (PAIRS == kHalves) {
      load8<BF16>(row + other * (BF16 ? 2 : 4), o);
    } else if constexpr (PAIRS == kHalvesOdd) {
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = load_elem<BF16>(row, place(j));
    }
  }
  __device__ __forceinline__ void other_weights(const void* w, bool w_bf16, float (&o)[8]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int at = PAIRS == kHalves ? other + j : place(j);
      o[j] = !w || !turns ? 1.0f : w_bf16 ? bf16_low(static_cast<const uint16_t*>(w)[at]) : static_cast<const float*>(w)[at];
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

__device__ __forceinline__ void lane_weights(const void* w, bool w_bf16, int d0, bool live, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    v[j] = !w || !live ? 1.0f : w_bf16 ? bf16_low(static_cast<const uint16_t*>(w)[d0 + j]) : static_cast<const float*>(w)[d0 + j];
}

// Cosines and sines of tokens first .. first + count - 1 into shared memory.
__device__ __forceinline__ void fill_table(const RotateArgs& a, int64_t first, int count, float2* table) {
  const int half = a.rotary_dim / 2;
  for (int i = threadIdx.x; i < count * half; i += kThreads) {
    const double turns = static_cast<double>(index_at(a.positions, a.position_bytes, first + i / half)) *
                         (static_cast<double>(a.freqs[i % half]) * 0.3183098861837906715);  // half turns
    double s, c;
    sincospi(turns, &s, &c);
    const float2 cs = make_float2(static_cast<float>(c), static_cast<float>(s));
    table[i] = cs;
    wait_lds_writes();
    hold_value(cs.x);
    hold_value(cs.y);
  }
  __syncthreads();
}

// A block takes `tokens` tokens from blockIdx.x * tokens on and of each the
// heads (queries', keys', values') blockIdx.y * heads .. + heads - 1.
template <bool BF16, int L, int PAIRS>
__global__ void __launch_bounds__(kThreads) rotate_kernel(RotateArgs a, int tokens, int heads) {
  constexpr int kElem = BF16 ? 2 : 4, kTeams = kThreads / L;
  __shared__ __attribute__((aligned(16))) float2 table[kTable];
  const LanePart<PAIRS> lane(threadIdx.x % L, a.head_dim, a.rotary_dim);
  const int total = a.q_heads + a.kv_heads * (a.v.data ? 2 : 1);
  const int h0 = blockIdx.y * heads, nh = total - h0 < heads ? total - h0 : heads;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tokens;
  const int nt = a.n - t0 < tokens ? static_cast<int>(a.n - t0) : tokens, half = a.rotary_dim / 2;
  float qw[8], kw[8], qo[8], ko[8];
  lane_weights(a.q_weight, a.w_bf16, lane.d0, lane.live, qw);
  lane_weights(a.k_weight, a.w_bf16, lane.d0, lane.live, kw);
  if constexpr (PAIRS != kNeighbours) {
    lane.other_weights(a.q_weight, a.w_bf16, qo);
    lane.other_weights(a.k_weight, a.w_bf16, ko);
  }
  if (h0 < a.q_heads + a.kv_heads) fill_table(a, t0, nt, table);

  for (int i = threadIdx.x / L; i < nt * nh; i += kTeams) {
    const int t = i / nh;
    int h = h0 + i % nh;
    const int64_t token = t0 + t;
    const bool is_q = h < a.q_heads, is_v = h >= a.q_heads + a.kv_heads;
    const HeadRows& from = is_q ? a.q : is_v ? a.v : a.k;
    const HeadRows& to = is_q ? a.q_out : is_v ? a.v_out : a.k_out;
    h -= is_q ? 0 : is_v ? a.q_heads + a.kv_heads : a.q_heads;
    int64_t out_row = token;
    if (a.slots && !is_q) {
      out_row = index_at(a.slots, a.slot_bytes, token);
      if (out_row < 0 || out_row >= a.cache_rows) continue;  // a whole team
    }
    const uint8_t* const x_row = from.data + (token * from.row + h * from.head) * kElem;
    float y[8] = {0.0f}, o[8] = {0.0f};
    if (lane.live) load8<BF16>(x_row + lane.d0 * kElem, y);
    if (!is_v) {
      if (lane.turns) lane.template load_others<BF16>(x_row, o);
      if (a.norm) {
        float ss = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = __builtin_fmaf(y[j], y[j], ss);
        const float r = rsqrtf(team_sum<L>(ss) / static_cast<float>(a.head_dim) + a.eps);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          y[j] *= r * (is_q ? qw[j] : kw[j]);
          if constexpr (PAIRS != kNeighbours) o[j] *= r * (is_q ? qo[j] : ko[j]);
        }
      }
      if (lane.turns) lane.template turn<false>(y, o, table + t * half);
    }
    if (lane.live) store8<BF16>(to.data + (out_row * to.row + h * to.head + lane.d0) * kElem, y);
  }
}

// The gradient's blocks walk over chunks of tokens; the shares of the weights'
// gradients stay in registers until the last one.
template <bool BF16, int L, int PAIRS>
__global__ void __launch_bounds__(kThreads) rotate_grad_kernel(RotateArgs a, int tokens, int64_t chunks) {
  constexpr int kElem = BF16 ? 2 : 4, kTeams = kThreads / L;
  __shared__ __attribute__((aligned(16))) float2 table[kTable];
  const int part = threadIdx.x % L;
  const LanePart<PAIRS> lane(part, a.head_dim, a.rotary_dim);
  const int heads = a.q_heads + a.kv_heads, half = a.rotary_dim / 2;
  float qw[8], kw[8], dqw[8], dkw[8];
  lane_weights(a.q_weight, a.w_bf16, lane.d0, lane.live, qw);
  lane_weights(a.k_weight, a.w_bf16, lane.d0, lane.live, kw);
#pragma unroll
  for (int j = 0; j < 8; ++j) dqw[j] = dkw[j] = 0.0f;

  for (int64_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int64_t t0 = c * tokens;
    const int nt = a.n - t0 < tokens ? static_cast<int>(a.n - t0) : tokens;
    __syncthreads();  // the last chunk's table is read
    fill_table(a, t0, nt, table);
    for (int i = threadIdx.x / L; i < nt * heads; i += kTeams) {
      const int t = i / heads;
      int h = i % heads;
      const int64_t token = t0 + t;
      const bool is_q = h < a.q_heads;
      const HeadRows& from = is_q ? a.q : a.k;
      const HeadRows& grad = is_q ? a.dq : a.dk;
      const HeadRows& to = is_q ? a.q_out : a.k_out;
      h -= is_q ? 0 : a.q_heads;
      const uint8_t* const g_row = grad.data + (token * grad.row + h * grad.head) * kElem;
      float u[8] = {0.0f}, o[8] = {0.0f};
      if (lane.live) load8<BF16>(g_row + lane.d0 * kElem, u);
      if (lane.turns) {
        lane.template load_others<BF16>(g_row, o);
        lane.template turn<true>(u, o, table + t * half);
      }
      if (a.norm) {
        float x[8] = {0.0f}, ss = 0.0f, dot = 0.0f;
        if (lane.live) load8<BF16>(from.data + (token * from.row + h * from.head + lane.d0) * kElem, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          ss = __builtin_fmaf(x[j], x[j], ss);
          dot = __builtin_fmaf(u[j] * (is_q ? qw[j] : kw[j]), x[j], dot);
        }
        const float n = static_cast<float>(a.head_dim), r = rsqrtf(team_sum<L>(ss) / n + a.eps), k = r * (team_sum<L>(dot) / n);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float xr = x[j] * r, g = u[j];
          u[j] = r * __builtin_fmaf(-xr, k, g * (is_q ? qw[j] : kw[j]));
          if (is_q)
            dqw[j] = __builtin_fmaf(g, xr, dqw[j]);
          else
            dkw[j] = __builtin_fmaf(g, xr, dkw[j]);
        }
      }
      if (lane.live) store8<BF16>(to.data + (token * to.row + h * to.head + lane.d0) * kElem, u);
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
  if (d < head_dim)
    for (int b = r * each; b < end; ++b) sum += part[(static_cast<int64_t>(b) * 2 + which) * head_dim + d];
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

// Tokens of a block: heads enough for each team to take up to four, fewer
// while that leaves compute units idle.
int tokens_of(int64_t n, int heads, int head_dim) {
  const int teams = kThreads / lanes_of(head_dim);
  const int64_t items = ceil_div(n * heads, 4 * kCus);
  const int64_t each = items < teams ? teams : items > 4 * teams ? 4 * teams : items;
  const int64_t tokens = each / heads;
  return static_cast<int>(tokens < 1 ? 1 : tokens > n ? n : tokens);
}

// Heads of a block: all, or one token's heads over several blocks while there
// are few tokens.
int heads_of(int64_t n, int total, int tokens, int head_dim) {
  const int teams = kThreads / lanes_of(head_dim);
  return tokens == 1 && n * ceil_div(total, teams) <= 8 * kCus ? teams : total;
}

template <bool BF16, int L, int PAIRS>
hipError_t launch_at(const RotateArgs& a, hipStream_t s) {
  const int total = a.q_heads + a.kv_heads * (a.v.data ? 2 : 1);
  const int tokens = tokens_of(a.n, total, a.head_dim);
  const int heads = heads_of(a.n, total, tokens, a.head_dim);
  rotate_kernel<BF16, L, PAIRS><<<dim3(static_cast<uint32_t>(ceil_div(a.n, tokens)), static_cast<uint32_t>(ceil_div(total, heads))),
                                  dim3(kThreads), 0, s>>>(a, tokens, heads);
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

int64_t rotate_blocks(int64_t n, int q_heads, int kv_heads, bool values, int head_dim) {
  const int total = q_heads + kv_heads * (values ? 2 : 1), tokens = tokens_of(n, total, head_dim);
  return ceil_div(n, tokens) * ceil_div(total, heads_of(n, total, tokens, head_dim));
}

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
