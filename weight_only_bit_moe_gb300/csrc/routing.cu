// Routing and its balance (moe_routing.h): the experts of each token, the pairs of
// each expert, the balance loss and the gradients by the logits.
//
// A warp owns a token.  Lane l holds the experts (32 i + l) V .. + V - 1 for i = 0,
// 1, ..: V = 4 where the rows allow vector loads, so a token of 128 experts is one
// load of a lane.  PER registers a lane serve up to 32 PER experts.
#include "products_tc.cuh"
#include "../../include/moe_routing.h"

namespace moe {

constexpr int kRtThreads = 256, kRtWarps = kRtThreads / 32;
constexpr int kRtSequences = 1 << 20;
// The counter of the last CTA of a loss, behind those of the products' tiles.
constexpr int kRtCounter = kProdCounterBytes / 4 - 1;
static_assert(kRtCounter >= kProdPartials, "a product's counter");

struct RouteArgs {
  const void* logits;
  int64_t ld;
  const float* bias;
  int tokens, E, k, score, renorm;
  float scale;
  float* weights;
  int32_t* ids;
  const float* dw;       // gradient
  int64_t dw_ld;
  const int32_t* in_ids;
  void* out;
  int64_t out_ld;
};

// ---------------------------------------------------------------- values
// Order of floats as unsigned numbers: -infinity is above 0, which stands for no value.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);  // (-0 counts as 0)
  return b ^ (b >> 31 ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ (k >> 31 ? 0x80000000u : 0xFFFFFFFFu));
}
__device__ __forceinline__ float warp_max(float v) {
  return key_value(__reduce_max_sync(0xffffffffu, order_key(v)));
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// sigmoid(l) / exp(min(top, 0)), top at least the largest l: in range where the sigmoids themselves are not.
__device__ __forceinline__ float shifted_sigmoid(float l, float floor) {
  return __fdividef(expf(fminf(l, 0.0f) - floor), 1.0f + expf(-fabsf(l)));
}
__device__ __forceinline__ float sigmoid(float l) {
  const float u = expf(-fabsf(l));
  return (l >= 0.0f ? 1.0f : u) / (1.0f + u);
}
// What is subtracted before exponentials: the largest value, or 0 for a token of -infinities.
__device__ __forceinline__ float finite_or_0(float v) { return v == -INFINITY ? 0.0f : v; }

template <int V>
__device__ __forceinline__ int expert_of(int i, int lane) {
  return ((i / V) * 32 + lane) * V + i % V;
}

// A token's logits, -infinity past the last.  V = 4: rows on a boundary of four elements, E a multiple of four.
template <int TYPE, int PER, int V>
__device__ __forceinline__ void load_row(const void* base, int64_t row_at, int E, int lane, float (&v)[PER]) {
#pragma unroll
  for (int i = 0; i < PER; i += V) {
    const int e = expert_of<V>(i, lane);
    if constexpr (V == 1) {
      v[i] = e < E ? load_elem(base, row_at + e, TYPE) : -INFINITY;
    } else if (e >= E) {
      v[i] = v[i + 1] = v[i + 2] = v[i + 3] = -INFINITY;
    } else if (TYPE == kFp32) {
      const float4 f = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + row_at + e);
      v[i] = f.x, v[i + 1] = f.y, v[i + 2] = f.z, v[i + 3] = f.w;
    } else {
      const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + row_at + e);
      const uint32_t w[2] = {u.x, u.y};
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (TYPE == kBf16) {
          v[i + 2 * j] = __uint_as_float(w[j] << 16);
          v[i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        } else {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
          v[i + 2 * j] = f.x;
          v[i + 2 * j + 1] = f.y;
        }
      }
    }
  }
}
template <int TYPE, int PER, int V>
__device__ __forceinline__ void store_row(void* base, int64_t row_at, int E, int lane, const float (&v)[PER]) {
#pragma unroll
  for (int i = 0; i < PER; i += V) {
    const int e = expert_of<V>(i, lane);
    if (e >= E) continue;
    if constexpr (V == 1) {
      store_elem(base, row_at + e, TYPE, v[i]);
    } else if (TYPE == kFp32) {
      *reinterpret_cast<float4*>(static_cast<float*>(base) + row_at + e) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    } else {
      const uint2 u = TYPE == kBf16 ? make_uint2(pack_bf16x2(v[i], v[i + 1]), pack_bf16x2(v[i + 2], v[i + 3]))
                                    : make_uint2(pack_half2(v[i], v[i + 1]), pack_half2(v[i + 2], v[i + 3]));
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(base) + row_at + e) = u;
    }
  }
}

// ---------------------------------------------------------------- choice
// The choice of a token whose p + bias lie too close for 32 bits, from its logits
// again: lane j gets the j-th expert or -1.
__device__ __noinline__ int choose_in_64(const RouteArgs& a, int type, int64_t row_at, int lane) {
  double key[32];
  double top = -INFINITY, z = 0.0;
  if (a.score == MOE_SCORE_SOFTMAX) {
#pragma unroll 1
    for (int e = lane; e < a.E; e += 32) top = fmax(top, (double)load_elem(a.logits, row_at + e, type));
    for (int o = 16; o > 0; o >>= 1) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, o));
#pragma unroll 1
    for (int e = lane; e < a.E; e += 32) z += exp((double)load_elem(a.logits, row_at + e, type) - top);
    z = warp_sum(z);
  }
#pragma unroll 1
  for (int i = 0; i < 32; ++i) {
    const int e = lane + 32 * i;
    key[i] = -INFINITY;
    if (e >= a.E) continue;
    const double l = load_elem(a.logits, row_at + e, type);
    if (l == -INFINITY) continue;
    double p;
    if (a.score == MOE_SCORE_SOFTMAX) {
      p = exp(l - top) / z;
    } else {
      const double u = exp(-fabs(l));
      p = (l >= 0.0 ? 1.0 : u) / (1.0 + u);
    }
    key[i] = p + (double)a.bias[e];
  }
  int mine = -1;
#pragma unroll 1
  for (int j = 0; j < a.k; ++j) {
    double best = -INFINITY;
    int at = 1 << 30;
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (key[i] > best) {
        best = key[i];
        at = lane + 32 * i;
      }
    for (int o = 16; o > 0; o >>= 1) {
      const double other = __shfl_xor_sync(0xffffffffu, best, o);
      const int other_at = __shfl_xor_sync(0xffffffffu, at, o);
      if (other > best || (other == best && other_at < at)) {
        best = other;
        at = other_at;
      }
    }
    if (best == -INFINITY) break;
    if (lane == j) mine = at;
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (lane + 32 * i == at) key[i] = -INFINITY;
  }
  return mine;
}

template <int TYPE, int PER, int V>
__global__ void __launch_bounds__(kRtThreads) route_kernel(const __grid_constant__ RouteArgs a) {
  grid_dependents_launch();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const int64_t token = (int64_t)blockIdx.x * kRtWarps + (threadIdx.x >> 5);
  if (token >= a.tokens) return;
  const bool softmax = a.score == MOE_SCORE_SOFTMAX;
  float v[PER];
  load_row<TYPE, PER, V>(a.logits, token * a.ld, a.E, lane, v);
  float most = v[0];  // (NaN passes on)
#pragma unroll
  for (int i = 1; i < PER; ++i) most = fmax_nan(most, v[i]);
  bool bad = !(most < INFINITY);
  const float top = warp_max(most);
  const float shift = finite_or_0(top);
  // softmax: the sum over all experts, where a weight or a key needs it
  float z = 1.0f;
  if (softmax && (a.bias || !a.renorm)) {
    z = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) z += expf(v[i] - shift);
    z = warp_sum(z);
  }
  uint32_t key[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    float c = v[i];
    if (a.bias) {
      const int e = expert_of<V>(i, lane);
      if (e < a.E) {
        const float b = __ldg(a.bias + e);
        bad |= !(b < INFINITY);
        if (c != -INFINITY) c = (softmax ? expf(c - shift) / z : sigmoid(c)) + b;
      }
    }
    key[i] = c == -INFINITY ? 0u : order_key(c);
  }
  int32_t* ids = a.ids + token * a.k;
  float* weights = a.weights + token * a.k;
  if (__any_sync(0xffffffffu, bad)) {
    if (lane < a.k) {
      ids[lane] = -1;
      weights[lane] = __uint_as_float(0x7FC00000u);
    }
    return;
  }
  // The largest key k times over, and with a bias once more: a 32-bit p is off by at
  // most 2^-17 of the largest p (softmax: the exponentials' and the sum's rounding;
  // p |ln p| < 1/e keeps the difference's small) or 2^-20 (sigmoid), the sum with the
  // bias by 2^-24 of itself, so keys further apart than twice that are in order.
  const float slack = !a.bias ? 0.0f : softmax ? 7.6293945e-6f / z : 9.5367432e-7f;
  const int rounds = a.bias ? min(a.k + 1, a.E) : a.k;
  int mine = -1;
  float picked = 0.0f, before = 0.0f;
  bool close = false;
  for (int j = 0; j < rounds; ++j) {
    uint32_t local = key[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) local = max(local, key[i]);
    const uint32_t best = __reduce_max_sync(0xffffffffu, local);
    if (best == 0u) break;
    const float now = key_value(best);
    if (a.bias) {
      if (j > 0 && before - now <= 2.0f * slack + 2.3841858e-7f * fmaxf(fabsf(before), fabsf(now))) close = true;
      before = now;
      if (j == a.k) break;
    }
    int at = 1 << 30;
#pragma unroll
    for (int i = PER - 1; i >= 0; --i)
      if (key[i] == best) at = expert_of<V>(i, lane);
    at = __reduce_min_sync(0xffffffffu, at);
    float logit = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (expert_of<V>(i, lane) == at) {
        key[i] = 0u;
        logit = v[i];
      }
    logit = __shfl_sync(0xffffffffu, logit, (at / V) % 32);
    if (lane == j) {
      mine = at;
      picked = logit;
    }
  }
  if (close) {
    mine = choose_in_64(a, TYPE, token * a.ld, lane);
    if (mine >= 0) picked = load_elem(a.logits, token * a.ld + mine, TYPE);
  }
  float w = 0.0f;
  if (softmax) {
    if (a.renorm) {
      const float first = finite_or_0(warp_max(mine >= 0 ? picked : -INFINITY));
      if (mine >= 0) w = expf(picked - first);
    } else if (mine >= 0) {
      w = expf(picked - shift) / z;
    }
  } else if (a.renorm) {
    const float floor = fminf(finite_or_0(warp_max(mine >= 0 ? picked : -INFINITY)), 0.0f);
    if (mine >= 0) w = shifted_sigmoid(picked, floor);
  } else if (mine >= 0) {
    w = sigmoid(picked);
  }
  if (a.renorm) {
    const float sum = warp_sum(w);
    if (mine >= 0) w = w / sum;
  }
  if (lane < a.k) {
    ids[lane] = mine;
    weights[lane] = mine >= 0 ? a.scale * w : 0.0f;
  }
}

// Gradient by the logits, with g the gradient by the weights, c scale and sums over the chosen:
//   softmax, renormalised   dl_j = w_j (g_j - sum g w / c)
//   softmax                 dl_e = c p_e ([e chosen] g_e - sum g p)
//   sigmoid, renormalised   dl_j = w_j (g_j - sum g w / c) (1 - p_j)
//   sigmoid                 dl_j = c g_j p_j (1 - p_j)
// Only the softmax over all experts reads the row; the others read the chosen logits.
template <int TYPE, int PER, int V>
__global__ void __launch_bounds__(kRtThreads) route_grad_kernel(const __grid_constant__ RouteArgs a) {
  grid_dependents_launch();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const int64_t token = (int64_t)blockIdx.x * kRtWarps + (threadIdx.x >> 5);
  if (token >= a.tokens) return;
  const bool softmax = a.score == MOE_SCORE_SOFTMAX;
  int id = -1;
  float g = 0.0f, l = -INFINITY;
  if (lane < a.k) {
    id = a.in_ids[token * a.k + lane];
    if (id < 0 || id >= a.E) id = -1;
    if (id >= 0) {
      g = a.dw[token * a.dw_ld + lane];
      l = load_elem(a.logits, token * a.ld + id, TYPE);
    }
  }
  float out[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) out[i] = 0.0f;
  float part = 0.0f;  // what the lane's slot adds to its expert
  if (__any_sync(0xffffffffu, id >= 0)) {
    if (softmax && !a.renorm) {
      float v[PER];
      load_row<TYPE, PER, V>(a.logits, token * a.ld, a.E, lane, v);
      float most = v[0];
#pragma unroll
      for (int i = 1; i < PER; ++i) most = fmaxf(most, v[i]);
      const float shift = finite_or_0(warp_max(most));
      float z = 0.0f;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        v[i] = expf(v[i] - shift);
        z += v[i];
      }
      z = warp_sum(z);
      const float p = id >= 0 ? expf(l - shift) / z : 0.0f;
      const float mean = warp_sum(g * p), c = a.scale;
      part = c * p * g;
#pragma unroll
      for (int i = 0; i < PER; ++i) out[i] = -c * (v[i] / z) * mean;
    } else if (a.renorm) {
      const float first = finite_or_0(warp_max(l));
      const float e = id < 0 ? 0.0f : softmax ? expf(l - first) : shifted_sigmoid(l, fminf(first, 0.0f));
      const float sum = warp_sum(e);
      const float w = sum > 0.0f || sum != sum ? e / sum : 0.0f;
      const float mean = warp_sum(g * w);
      part = a.scale * w * (g - mean);
      if (!softmax) part *= sigmoid(-l);
    } else {
      part = a.scale * g * sigmoid(l) * sigmoid(-l);
    }
    if (id < 0) part = 0.0f;
    for (int j = 0; j < a.k; ++j) {
      const int at = __shfl_sync(0xffffffffu, id, j);
      const float add = __shfl_sync(0xffffffffu, part, j);
      if (at < 0) continue;
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (expert_of<V>(i, lane) == at) out[i] += add;
    }
  }
  store_row<TYPE, PER, V>(a.out, token * a.out_ld, a.E, lane, out);
}

// ---------------------------------------------------------------- counts
struct CountArgs {
  const int32_t* ids;
  int64_t ld;
  int tokens, k, S, E;
  const int32_t* offsets;
  int32_t* counts;
  unsigned* status;
};

// Tokens [r0, r1) of sequence s, inside [0, tokens] whatever the offsets hold.
__device__ __forceinline__ void sequence_rows(const int32_t* offsets, int s, int tokens, int& r0, int& r1) {
  if (!offsets) {
    r0 = 0;
    r1 = tokens;
    return;
  }
  r0 = min(max(__ldg(offsets + s), 0), tokens);
  r1 = max(r0, min(max(__ldg(offsets + s + 1), 0), tokens));
}
__device__ __forceinline__ bool sequence_bad(const int32_t* offsets, int s, int tokens) {
  if (!offsets) return false;
  const int a = __ldg(offsets + s), b = __ldg(offsets + s + 1);
  return a < 0 || b < a || b > tokens;
}

constexpr int kCtThreads = 512, kCtCopies = 4;

// A cluster per sequence.  Each CTA counts its part of the ids in shared memory, in
// four copies by lane so that popular experts collide less; then each CTA adds up
// its part of the experts over the cluster and writes it: integers, in any order.
__global__ void __launch_bounds__(kCtThreads) count_kernel(const __grid_constant__ CountArgs a) {
  __shared__ int32_t hist[kCtCopies][kProdGroups];
  const int tid = threadIdx.x;
  uint32_t rank, width;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(width));
  const int s = blockIdx.x / width;
  for (int i = tid; i < kCtCopies * kProdGroups; i += kCtThreads) (&hist[0][0])[i] = 0;
  grid_dependents_launch();
  grid_dependency_wait();
  int r0, r1;
  sequence_rows(a.offsets, s, a.tokens, r0, r1);
  if (tid == 0 && rank == 0 && sequence_bad(a.offsets, s, a.tokens)) atomicOr(a.status, kStatusRouting);
  __syncthreads();
  const int pairs = (r1 - r0) * a.k;
  const bool dense = a.ld == a.k;
  const int32_t* ids = a.ids + r0 * a.ld;
  for (int64_t p = (int64_t)rank * kCtThreads + tid; p < pairs; p += (int64_t)width * kCtThreads) {
    const int id = dense ? ids[p] : ids[p / a.k * a.ld + p % a.k];
    if (id >= 0 && id < a.E) atomicAdd(&hist[tid % kCtCopies][id], 1);
  }
  __syncthreads();
  for (int e = tid; e < a.E; e += kCtThreads) {
    int sum = 0;
#pragma unroll
    for (int c = 0; c < kCtCopies; ++c) sum += hist[c][e];
    hist[0][e] = sum;
  }
  cluster_sync_all();
  for (int e = rank * kCtThreads + tid; e < a.E; e += width * kCtThreads) {
    int sum = 0;
    for (uint32_t c = 0; c < width; ++c) {
      int32_t n;
      asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(n) : "r"(map_to_rank(smem_u32(&hist[0][e]), c)) : "memory");
      sum += n;
    }
    a.counts[(int64_t)s * a.E + e] = sum;
  }
  cluster_sync_all();  // (nobody leaves while its counts are read)
}

// ---------------------------------------------------------------- balance
struct BalanceArgs {
  const void* logits;
  int64_t ld;
  int tokens, E, S, score;
  const int32_t* counts;
  const int32_t* offsets;
  float* loss;
  const float* dloss;    // gradient
  void* out;
  int64_t out_ld;
  unsigned* status;
  int32_t* counter;
  float* partial;        // [warps + S]: warp w, sequence s at w + s
  int rows_per_warp;
};

// The sequence of a token, from the first one that may hold it on; S: none.
struct SequenceWalk {
  int s, r0, r1;
  __device__ __forceinline__ void start(const BalanceArgs& a, int token) {
    int lo = 0, hi = a.S;  // the first sequence that ends past the token
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      int b0, b1;
      sequence_rows(a.offsets, mid, a.tokens, b0, b1);
      if (b1 > token) hi = mid;
      else lo = mid + 1;
    }
    s = lo;
    if (s < a.S) sequence_rows(a.offsets, s, a.tokens, r0, r1);
  }
  // On to the sequence that ends past the token; true where it is another one.
  __device__ __forceinline__ bool reach(const BalanceArgs& a, int token) {
    bool moved = false;
    while (s < a.S && r1 <= token) {
      ++s;
      moved = true;
      if (s < a.S) sequence_rows(a.offsets, s, a.tokens, r0, r1);
    }
    return moved;
  }
};

// Counts of the sequence, times num_experts / (C T).
template <int PER, int V>
__device__ __forceinline__ void load_counts(const BalanceArgs& a, const SequenceWalk& q, int lane, float (&c)[PER]) {
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = expert_of<V>(i, lane);
    c[i] = e < a.E ? (float)a.counts[(int64_t)q.s * a.E + e] : 0.0f;
    sum += c[i];
  }
  sum = warp_sum(sum) * (q.r1 - q.r0);
  const float factor = sum > 0.0 ? (float)(a.E / sum) : 0.0f;
#pragma unroll
  for (int i = 0; i < PER; ++i) c[i] *= factor;
}

// p of a token in v's place (times z), returns 1 / z; `rest` gets 1 - sigmoid.
template <int PER>
__device__ __forceinline__ float probabilities(float (&v)[PER], bool softmax, float* rest) {
  float most = v[0];
#pragma unroll
  for (int i = 1; i < PER; ++i) most = fmaxf(most, v[i]);
  const float shift = finite_or_0(warp_max(most)), floor = fminf(shift, 0.0f);
  float z = 0.0f;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (softmax) {
      v[i] = expf(v[i] - shift);
    } else {
      const float u = expf(-fabsf(v[i])), inv = __fdividef(1.0f, 1.0f + u);
      if (rest) rest[i] = (v[i] >= 0.0f ? u : 1.0f) * inv;
      v[i] = expf(fminf(v[i], 0.0f) - floor) * inv;
    }
    z += v[i];
  }
  z = warp_sum(z);
  return z == 0.0f ? 0.0f : 1.0f / z;
}

template <int TYPE, int PER, int V>
__global__ void __launch_bounds__(kRtThreads) balance_kernel(const __grid_constant__ BalanceArgs a) {
  __shared__ int last;
  const int lane = threadIdx.x & 31, warp = blockIdx.x * kRtWarps + (threadIdx.x >> 5);
  grid_dependents_launch();
  grid_dependency_wait();
  if (a.offsets)
    for (int s = blockIdx.x * kRtThreads + threadIdx.x; s < a.S; s += gridDim.x * kRtThreads)
      if (sequence_bad(a.offsets, s, a.tokens)) atomicOr(a.status, kStatusRouting);
  const int64_t first = (int64_t)warp * a.rows_per_warp;
  const int end = (int)min((int64_t)a.tokens, first + a.rows_per_warp);
  if (first < end) {
    SequenceWalk q;
    q.start(a, (int)first);
    float c[PER], sum = 0.0f;
    bool have = false;
    for (int token = (int)first; token < end; ++token) {
      const int old = q.s;
      if (q.reach(a, token)) {
        if (have && lane == 0) a.partial[warp + old] = sum;
        have = false;
        sum = 0.0f;
      }
      if (q.s == a.S) break;
      if (token < q.r0) continue;
      if (!have) load_counts<PER, V>(a, q, lane, c);
      have = true;
      float v[PER], inner = 0.0f;
      load_row<TYPE, PER, V>(a.logits, token * a.ld, a.E, lane, v);
      const float inv = probabilities<PER>(v, a.score == MOE_SCORE_SOFTMAX, nullptr);
#pragma unroll
      for (int i = 0; i < PER; ++i) inner = fmaf(v[i], c[i], inner);
      sum += warp_sum(inner) * inv;
    }
    if (have && lane == 0) a.partial[warp + q.s] = sum;
  }
  __syncthreads();
  if (threadIdx.x == 0) last = slice_arrive_last(a.counter, gridDim.x);
  __syncthreads();
  if (!last) return;
  // the last CTA: a warp per sequence adds the warps' parts in their order
  for (int s = threadIdx.x >> 5; s < a.S; s += kRtWarps) {
    int r0, r1;
    sequence_rows(a.offsets, s, a.tokens, r0, r1);
    double sum = 0.0;
    if (r0 < r1)
      for (int w = r0 / a.rows_per_warp + lane; w <= (r1 - 1) / a.rows_per_warp; w += 32)
        sum += *(volatile float*)(a.partial + w + s);
    sum = warp_sum(sum);
    if (lane == 0) a.loss[s] = (float)sum;
  }
}

// dl_e = dloss p_e (c_e - sum c p), c the counts times num_experts / (C T); sigmoid: p_e (1 - sigmoid_e) in
// the place of p_e.
template <int TYPE, int PER, int V>
__global__ void __launch_bounds__(kRtThreads) balance_grad_kernel(const __grid_constant__ BalanceArgs a) {
  const int lane = threadIdx.x & 31, warp = blockIdx.x * kRtWarps + (threadIdx.x >> 5);
  grid_dependents_launch();
  grid_dependency_wait();
  if (a.offsets)
    for (int s = blockIdx.x * kRtThreads + threadIdx.x; s < a.S; s += gridDim.x * kRtThreads)
      if (sequence_bad(a.offsets, s, a.tokens)) atomicOr(a.status, kStatusRouting);
  const int64_t first = (int64_t)warp * a.rows_per_warp;
  const int end = (int)min((int64_t)a.tokens, first + a.rows_per_warp);
  if (first >= end) return;
  const bool softmax = a.score == MOE_SCORE_SOFTMAX;
  SequenceWalk q;
  q.start(a, (int)first);
  float c[PER], dloss = 0.0f;
  bool have = false;
  for (int token = (int)first; token < end; ++token) {
    if (q.reach(a, token)) have = false;
    float v[PER];
    if (q.s == a.S || token < q.r0) {
#pragma unroll
      for (int i = 0; i < PER; ++i) v[i] = 0.0f;
    } else {
      if (!have) {
        load_counts<PER, V>(a, q, lane, c);
        dloss = a.dloss[q.s];
        have = true;
      }
      float rest[PER], inner = 0.0f;
      load_row<TYPE, PER, V>(a.logits, token * a.ld, a.E, lane, v);
      const float inv = probabilities<PER>(v, softmax, rest);
#pragma unroll
      for (int i = 0; i < PER; ++i) inner = fmaf(v[i], c[i], inner);
      inner = warp_sum(inner) * inv;
      const float g = dloss * inv;
#pragma unroll
      for (int i = 0; i < PER; ++i) v[i] = g * (softmax ? v[i] : v[i] * rest[i]) * (c[i] - inner);
    }
    store_row<TYPE, PER, V>(a.out, token * a.out_ld, a.E, lane, v);
  }
}

// ---------------------------------------------------------------- host
// The instance of KERNEL for a type, a number of experts and the rows' alignment.
#define MOE_ROUTING_PICK_V(KERNEL, T, V)                                                  \
  (E <= 32 ? (const void*)KERNEL<T, (V == 4 ? 4 : 1), V>                                   \
           : E <= 64 ? (const void*)KERNEL<T, (V == 4 ? 4 : 2), V>                         \
                     : E <= 128 ? (const void*)KERNEL<T, 4, V>                             \
                                : E <= 256 ? (const void*)KERNEL<T, 8, V>                  \
                                           : E <= 512 ? (const void*)KERNEL<T, 16, V>      \
                                                      : (const void*)KERNEL<T, 32, V>)
#define MOE_ROUTING_PICK(KERNEL)                                                          \
  static const void* pick_##KERNEL(int type, int E, bool four) {                          \
    if (type == kBf16) return four ? MOE_ROUTING_PICK_V(KERNEL, kBf16, 4) : MOE_ROUTING_PICK_V(KERNEL, kBf16, 1); \
    if (type == kFp16) return four ? MOE_ROUTING_PICK_V(KERNEL, kFp16, 4) : MOE_ROUTING_PICK_V(KERNEL, kFp16, 1); \
    return four ? MOE_ROUTING_PICK_V(KERNEL, kFp32, 4) : MOE_ROUTING_PICK_V(KERNEL, kFp32, 1);                    \
  }
MOE_ROUTING_PICK(route_kernel)
MOE_ROUTING_PICK(route_grad_kernel)
MOE_ROUTING_PICK(balance_kernel)
MOE_ROUTING_PICK(balance_grad_kernel)

static int elem_bytes(int type) { return type == kFp32 ? 4 : 2; }
static bool on_elements(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
// Rows that four elements at a time can be read from (NULL: none to read).
static bool in_fours(const void* p, int64_t ld, int E, int type) {
  return !p || (E % 4 == 0 && ld % 4 == 0 && on_elements(p, 4 * elem_bytes(type)));
}
// (Below 128 experts four a lane leave most of the lanes without work, but the loads are fewer.)

static bool good_rows(const void* p, int64_t ld, int E, int type) { return p && ld >= E && on_elements(p, elem_bytes(type)); }
static bool good_logits(int type, int tokens, int E) {
  return type >= kBf16 && type <= kFp32 && tokens >= 0 && E >= 1 && E <= kProdGroups &&
         (int64_t)tokens * E < (int64_t)1 << 40;
}
static bool good_score(int score) { return score == MOE_SCORE_SOFTMAX || score == MOE_SCORE_SIGMOID; }

template <typename Args>
static int launch_routing(const void* kernel, int grid, const Args& a, void* stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kRtThreads);
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void* args[] = {const_cast<Args*>(&a)};
  return cudaLaunchKernelExC(&cfg, kernel, args) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

static int check_workspace(const void* workspace, int64_t bytes) {
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255)) return MOE_ERR_INVALID;
  return bytes < MOE_PRODUCTS_WORKSPACE_BYTES ? MOE_ERR_WORKSPACE : MOE_OK;
}

// Tokens a warp takes one after the other: one until the GPU is full four times over.
static int plan_balance(BalanceArgs& a, int* grid) {
  const int sms = prod_sm_count();
  if (sms <= 0) return MOE_ERR_CUDA;
  const int64_t warps = (int64_t)sms * 4 * kRtWarps;
  a.rows_per_warp = (int)((a.tokens + warps - 1) / warps);
  if (a.rows_per_warp < 1) a.rows_per_warp = 1;
  const int64_t used = ((int64_t)a.tokens + a.rows_per_warp - 1) / a.rows_per_warp;
  *grid = (int)((used + kRtWarps - 1) / kRtWarps);
  if (*grid < 1) *grid = 1;
  return MOE_OK;
}

static void set_balance_workspace(BalanceArgs& a, void* workspace) {
  uint8_t* w = static_cast<uint8_t*>(workspace);
  a.status = reinterpret_cast<unsigned*>(w);
  a.counter = reinterpret_cast<int32_t*>(w + 256) + kRtCounter;
  a.partial = reinterpret_cast<float*>(w + MOE_PRODUCTS_WORKSPACE_HEAD_BYTES);
}

}  // namespace moe

using namespace moe;

extern "C" int moe_route(int dtype, const void* logits, int64_t logits_stride, const float* bias, int tokens,
                         int num_experts, int top_k, int score, int renormalize, float scale, float* weights,
                         int32_t* ids, void* stream) {
  if (!good_logits(dtype, tokens, num_experts) || !good_score(score) || renormalize < 0 || renormalize > 1)
    return MOE_ERR_INVALID;
  if (top_k < 1 || top_k > num_experts || top_k > MOE_MAX_TOP_K || logits_stride < num_experts) return MOE_ERR_INVALID;
  if (tokens == 0) return MOE_OK;
  if (!good_rows(logits, logits_stride, num_experts, dtype) || !weights || !ids || !on_elements(weights, 4) ||
      !on_elements(ids, 4) || !on_elements(bias, 4))
    return MOE_ERR_INVALID;
  RouteArgs a{};
  a.logits = logits, a.ld = logits_stride, a.bias = bias, a.tokens = tokens, a.E = num_experts, a.k = top_k;
  a.score = score, a.renorm = renormalize, a.scale = scale, a.weights = weights, a.ids = ids;
  const bool four = in_fours(logits, logits_stride, num_experts, dtype);
  return launch_routing(pick_route_kernel(dtype, num_experts, four), (tokens - 1) / kRtWarps + 1, a, stream);
}

extern "C" int moe_route_grad(int dtype, const float* dweights, int64_t dweights_stride, const void* logits,
                              int64_t logits_stride, const int32_t* ids, int tokens, int num_experts, int top_k,
                              int score, int renormalize, float scale, void* dlogits, int64_t dlogits_stride,
                              void* stream) {
  if (!good_logits(dtype, tokens, num_experts) || !good_score(score) || renormalize < 0 || renormalize > 1)
    return MOE_ERR_INVALID;
  if (top_k < 1 || top_k > num_experts || top_k > MOE_MAX_TOP_K || dweights_stride < top_k ||
      logits_stride < num_experts || dlogits_stride < num_experts)
    return MOE_ERR_INVALID;
  if (tokens == 0) return MOE_OK;
  if (!good_rows(logits, logits_stride, num_experts, dtype) || !good_rows(dlogits, dlogits_stride, num_experts, dtype) ||
      !dweights || !ids || !on_elements(dweights, 4) || !on_elements(ids, 4))
    return MOE_ERR_INVALID;
  RouteArgs a{};
  a.logits = logits, a.ld = logits_stride, a.tokens = tokens, a.E = num_experts, a.k = top_k;
  a.score = score, a.renorm = renormalize, a.scale = scale, a.dw = dweights, a.dw_ld = dweights_stride;
  a.in_ids = ids, a.out = dlogits, a.out_ld = dlogits_stride;
  const bool four = in_fours(logits, logits_stride, num_experts, dtype) &&
                    in_fours(dlogits, dlogits_stride, num_experts, dtype);
  return launch_routing(pick_route_grad_kernel(dtype, num_experts, four), (tokens - 1) / kRtWarps + 1, a, stream);
}

extern "C" int moe_expert_counts(const int32_t* ids, int64_t ids_stride, int tokens, int top_k,
                                 const int32_t* offsets, int num_sequences, int num_experts, int32_t* counts,
                                 void* workspace, int64_t workspace_bytes, void* stream) {
  if (tokens < 0 || top_k < 1 || (int64_t)tokens * top_k >= (int64_t)1 << 31 || ids_stride < top_k) return MOE_ERR_INVALID;
  if (num_experts < 1 || num_experts > kProdGroups || num_sequences < 1 || num_sequences > kRtSequences)
    return MOE_ERR_INVALID;
  if (!offsets && num_sequences != 1) return MOE_ERR_INVALID;
  if (!counts || (tokens > 0 && !ids) || !on_elements(ids, 4) || !on_elements(counts, 4) || !on_elements(offsets, 4))
    return MOE_ERR_INVALID;
  const int rc = check_workspace(workspace, workspace_bytes);
  if (rc != MOE_OK) return rc;
  const int sms = prod_sm_count();
  if (sms <= 0) return MOE_ERR_CUDA;
  CountArgs a{};
  a.ids = ids, a.ld = ids_stride, a.tokens = tokens, a.k = top_k, a.S = num_sequences, a.E = num_experts;
  a.offsets = offsets, a.counts = counts, a.status = static_cast<unsigned*>(workspace);
  // CTAs to a sequence: as many as fill the GPU, with some thousand ids each
  int width = 1;
  while (width < 8 && 2 * width * num_sequences <= sms && (int64_t)tokens * top_k / num_sequences > 2 * width * kCtThreads)
    width *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)num_sequences * width);
  cfg.blockDim = dim3(kCtThreads);
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = width;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, count_kernel, a) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

static int check_balance(int dtype, const void* logits, int64_t ld, int tokens, int E, const int32_t* counts,
                         const int32_t* offsets, int S, int score, const void* workspace, int64_t bytes) {
  if (!good_logits(dtype, tokens, E) || !good_score(score) || S < 1 || S > kRtSequences || ld < E) return MOE_ERR_INVALID;
  if (!offsets && S != 1) return MOE_ERR_INVALID;
  if (tokens > 0 && !good_rows(logits, ld, E, dtype)) return MOE_ERR_INVALID;
  if (!counts || !on_elements(counts, 4) || !on_elements(offsets, 4)) return MOE_ERR_INVALID;
  return check_workspace(workspace, bytes);
}

extern "C" int moe_balance_loss(int dtype, const void* logits, int64_t logits_stride, int tokens, int num_experts,
                                const int32_t* counts, const int32_t* offsets, int num_sequences, int score,
                                float* loss, void* workspace, int64_t workspace_bytes, void* stream) {
  int rc = check_balance(dtype, logits, logits_stride, tokens, num_experts, counts, offsets, num_sequences, score,
                         workspace, workspace_bytes);
  if (rc != MOE_OK) return rc;
  if (!loss || !on_elements(loss, 4)) return MOE_ERR_INVALID;
  BalanceArgs a{};
  a.logits = logits, a.ld = logits_stride, a.tokens = tokens, a.E = num_experts, a.S = num_sequences, a.score = score;
  a.counts = counts, a.offsets = offsets, a.loss = loss;
  set_balance_workspace(a, workspace);
  int grid;
  if ((rc = plan_balance(a, &grid)) != MOE_OK) return rc;
  const bool four = in_fours(logits, logits_stride, num_experts, dtype);
  return launch_routing(pick_balance_kernel(dtype, num_experts, four), grid, a, stream);
}

extern "C" int moe_balance_loss_grad(int dtype, const float* dloss, const void* logits, int64_t logits_stride,
                                     int tokens, int num_experts, const int32_t* counts, const int32_t* offsets,
                                     int num_sequences, int score, void* dlogits, int64_t dlogits_stride,
                                     void* workspace, int64_t workspace_bytes, void* stream) {
  int rc = check_balance(dtype, logits, logits_stride, tokens, num_experts, counts, offsets, num_sequences, score,
                         workspace, workspace_bytes);
  if (rc != MOE_OK) return rc;
  if (dlogits_stride < num_experts) return MOE_ERR_INVALID;
  if (tokens == 0) return MOE_OK;
  if (!dloss || !on_elements(dloss, 4) || !good_rows(dlogits, dlogits_stride, num_experts, dtype)) return MOE_ERR_INVALID;
  BalanceArgs a{};
  a.logits = logits, a.ld = logits_stride, a.tokens = tokens, a.E = num_experts, a.S = num_sequences, a.score = score;
  a.counts = counts, a.offsets = offsets, a.dloss = dloss, a.out = dlogits, a.out_ld = dlogits_stride;
  set_balance_workspace(a, workspace);
  int grid;
  if ((rc = plan_balance(a, &grid)) != MOE_OK) return rc;
  const bool four = in_fours(logits, logits_stride, num_experts, dtype) &&
                    in_fours(dlogits, dlogits_stride, num_experts, dtype);
  return launch_routing(pick_balance_grad_kernel(dtype, num_experts, four), grid, a, stream);
}
