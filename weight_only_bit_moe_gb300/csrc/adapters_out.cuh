// The second launch of the adapters of many rows (the first: adapters_mid.cu):
//   out[r, q] = base[r, q] + scale[l] sum_j mid[i, j] S[l](q, j)
#pragma once

#include "adapters.cuh"

namespace moe {

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(addr)
               : "memory");
}

// Register-fed: a CTA holds 128 rows' mid as MMA operands, high and low 16-bit parts
// (fp16: of the row divided by a power of two that brings its largest value below
// 2^14), and walks over columns, 128 at a time.  S passes through shared memory in an
// order that leaves eight consecutive columns of a row in each lane: base comes
// straight from memory into the lane that adds to it, and the sum goes straight back,
// 16 bytes each and 64 of a row by four lanes.  Rows without an adapter are tiles
// whose sums are zero (none of them where out is base).
constexpr int kOuThreads = 256, kOuCols = 128;

template <int KS>  // steps of 16 ranks, at most
struct OutCfg {
  static constexpr bool kRegs = KS <= 4;            // mid's operands stay in registers
  static constexpr int kBuffers = KS <= 8 ? 2 : 1;  // of S
  static constexpr int kFwdPitch = (2 * KS + 1) * 16, kGradPitch = kOuCols * 2 + 16;  // odd in 16 bytes
  static constexpr int kSBytes = kOuCols * kFwdPitch > 16 * KS * kGradPitch ? kOuCols * kFwdPitch : 16 * KS * kGradPitch;
  static constexpr int kMidBytes = kRegs ? 0 : 8 * KS * 2 * 512;
  static constexpr int kAlloc = kBuffers * kSBytes + kMidBytes;
  static constexpr int kCtas = KS <= 4 ? 2 : 1;
  static_assert(kCtas * (kAlloc + (kAdAdapters + 1) * 4 + 1024) <= 227 * 1024, "shared memory over the SM's");
};

struct OutPlan {
  int tiles, before, from;  // tiles of adapters; positions [0, before) and [from, rows) have none
  int rest0, rest1;         // tiles of those
  int chunks, ranges;       // column chunks, cut into ranges
};

template <int TYPE, int KS, bool FWD>
__global__ void __launch_bounds__(kOuThreads, OutCfg<KS>::kCtas) adapter_out_kernel(const __grid_constant__ AdapterArgs a) {
  using C = OutCfg<KS>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ int start[kAdAdapters + 1];
  __shared__ int warp_tot[kOuThreads / 32];
  const uint32_t smem_s = smem_u32(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  grid_dependents_launch();
  grid_dependency_wait();
  plan_adapters<kAtRows, kOuThreads>(a.offsets, a.rows, a.L, start, warp_tot, a.status);
  const int S = *(volatile int*)a.plan;
  OutPlan pl;
  pl.tiles = start[a.L];
  pl.before = pl.from = pl.rest0 = pl.rest1 = 0;
  if (a.base != a.out) {
    pl.before = min(max(__ldg(a.offsets), 0), a.rows);
    pl.from = max(pl.before, min(max(__ldg(a.offsets + a.L), 0), a.rows));
    pl.rest0 = (pl.before + kAtRows - 1) / kAtRows;
    pl.rest1 = (a.rows - pl.from + kAtRows - 1) / kAtRows;
  }
  pl.chunks = (a.Q + kOuCols - 1) / kOuCols;
  const int tiles = pl.tiles + pl.rest0 + pl.rest1;
  {  // ranges of columns to a tile: the number that minimises rounds * (chunks of a range + 2), a lane per number
    const int n = lane + 1;
    uint32_t cost = 0xFFFFFFu;
    if (n <= pl.chunks) {
      const int64_t rounds = ((int64_t)tiles * n + gridDim.x - 1) / gridDim.x;
      cost = (uint32_t)min((int64_t)0xFFFFFF, rounds * ((pl.chunks + n - 1) / n + 2));
    }
    pl.ranges = (int)(__reduce_min_sync(0xffffffffu, cost * 64 + n) & 63);
  }
  const int64_t items = (int64_t)tiles * pl.ranges;
  const float* part = S == 1 ? a.mid : a.part;
  const int64_t slice = (int64_t)a.rows * a.R;
  const int steps = (a.R + 15) / 16;
  const uint16_t* base = static_cast<const uint16_t*>(a.base);
  uint16_t* out = static_cast<uint16_t*>(a.out);

  int l = 0;
  for (int64_t w = blockIdx.x; w < items; w += gridDim.x) {
    const int tile = (int)(w / pl.ranges), range = (int)(w - (int64_t)tile * pl.ranges);
    const int c0 = (int)((int64_t)range * pl.chunks / pl.ranges), c1 = (int)((int64_t)(range + 1) * pl.chunks / pl.ranges);
    int pos, n;
    const bool has = tile < pl.tiles;
    if (has) {
      while (start[l + 1] <= tile) ++l;
      int i0, i1;
      adapter_rows(a.offsets, a.rows, l, i0, i1);
      pos = i0 + (tile - start[l]) * kAtRows;
      n = min(kAtRows, i1 - pos);
    } else {
      const int k = tile - pl.tiles;
      pos = k < pl.rest0 ? k * kAtRows : pl.from + (k - pl.rest0) * kAtRows;
      n = min(kAtRows, (k < pl.rest0 ? pl.before : a.rows) - pos);
    }
    const uint16_t* s = static_cast<const uint16_t*>(a.s) + (has ? l * a.s_l : 0);

    // S of a chunk into buffer b
    auto fetch = [&](int chunk, int b) {
      if (!has) return;
      const uint32_t dst = smem_s + b * C::kSBytes;
      const int q0 = chunk * kOuCols;
      if (FWD) {
        for (int u = tid; u < kOuCols * 2 * steps; u += kOuThreads) {
          const int q = u / (2 * steps), c = u - q * 2 * steps;
          const int line = (q & ~31) + ((q >> 1) & 3) * 8 + ((q >> 3) & 3) * 2 + (q & 1);
          const bool in = q0 + q < a.Q && 8 * c < a.R;
          cp_async16(dst + line * C::kFwdPitch + c * 16, s + (in ? (q0 + q) * a.s_r + 8 * c : 0), in ? 16 : 0);
        }
      } else {
        for (int u = tid; u < 16 * steps * (kOuCols / 2); u += kOuThreads) {
          const int j = u / (kOuCols / 2), v = u % (kOuCols / 2);
          const bool in = q0 + 2 * v < a.Q && j < a.R;
          cp_async4(dst + j * C::kGradPitch + (v & ~15) * 4 + ((v & 3) * 4 + ((v >> 2) & 3)) * 4,
                    s + (in ? j * a.s_r + q0 + 2 * v : 0), in ? 4 : 0);
        }
      }
    };
    __syncthreads();  // the last item's reads of S are done
    if (C::kBuffers == 2) {
      fetch(c0, 0);
      cp_async_commit();
    }

    // rows 16 warp + g and + 8 of the tile, and their mid
    int row[2];
    float factor[2] = {1.0f, 1.0f};
    const float* m[2];
    bool held[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = 16 * warp + g + 8 * h;
      held[h] = at < n;
      row[h] = held[h] ? row_of(a.order, a.rows, pos + at, a.status) : -1;
      m[h] = part + (int64_t)(pos + (held[h] ? at : 0)) * a.R;
    }
    auto mid2 = [&](int h, int j) {
      float2 v = make_float2(0.0f, 0.0f);
      if (held[h] && j < a.R) {
        v = *reinterpret_cast<const float2*>(m[h] + j);
        for (int k = 1; k < S; ++k) {
          const float2 u = *reinterpret_cast<const float2*>(m[h] + k * slice + j);
          v.x += u.x;
          v.y += u.y;
        }
        if (S > 1 && a.want_mid && range == 0) *reinterpret_cast<float2*>(a.mid + (int64_t)(pos + 16 * warp + g + 8 * h) * a.R + j) = v;
      }
      return v;
    };
    uint32_t mh[C::kRegs ? KS : 1][4], ml[C::kRegs ? KS : 1][4];
    uint4* kept = reinterpret_cast<uint4*>(smem_raw + C::kBuffers * C::kSBytes) + warp * KS * 2 * 32;
    if (has) {
      if (TYPE == kFp16) {
        float top[2] = {0.0f, 0.0f};
        for (int ks = 0; ks < steps; ++ks)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int o = 0; o < 2; ++o) {
              const float2 v = mid2(h, 16 * ks + 8 * o + 2 * t);
              top[h] = fmaxf(top[h], fmaxf(fabsf(v.x), fabsf(v.y)));
            }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
          top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2));
          // 2^(exponent - 13), at least 2^-126: the largest value becomes 2^13 .. 2^14
          const int e = max((int)((__float_as_uint(top[h]) >> 23) & 255) - 13, 1);
          if (top[h] > 0.0f && top[h] < INFINITY) factor[h] = __uint_as_float((uint32_t)e << 23);
        }
      }
      const float inv[2] = {1.0f / factor[0], 1.0f / factor[1]};
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        if (ks >= steps) break;
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int o = 0; o < 2; ++o)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float2 v = mid2(h, 16 * ks + 8 * o + 2 * t);
            if (TYPE == kFp16) v.x *= inv[h], v.y *= inv[h];
            split_type<TYPE>(v.x, v.y, hi[2 * o + h], lo[2 * o + h]);
          }
        if (C::kRegs) {
#pragma unroll
          for (int u = 0; u < 4; ++u) mh[C::kRegs ? ks : 0][u] = hi[u], ml[C::kRegs ? ks : 0][u] = lo[u];
        } else {
          kept[(2 * ks) * 32 + lane] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          kept[(2 * ks + 1) * 32 + lane] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
      }
    }
    const float scale = has ? (a.scale ? a.scale[l] : 1.0f) : 0.0f;
    const float mul[2] = {scale * factor[0], scale * factor[1]};

    for (int chunk = c0; chunk < c1; ++chunk) {
      const int b = C::kBuffers == 2 ? (chunk - c0) & 1 : 0;
      const int q0 = chunk * kOuCols + 8 * t;
      uint4 was[kOuCols / 32][2];
#pragma unroll
      for (int u = 0; u < kOuCols / 32; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int q = q0 + 32 * u;
          was[u][h] = base && row[h] >= 0 && q < a.Q ? *reinterpret_cast<const uint4*>(base + (int64_t)row[h] * a.base_ld + q)
                                                     : make_uint4(0, 0, 0, 0);
        }
      if (C::kBuffers == 2) {
        if (chunk + 1 < c1) fetch(chunk + 1, b ^ 1);
        cp_async_commit();
        cp_async_wait<1>();
      } else {
        fetch(chunk, 0);
        cp_async_commit();
        cp_async_wait<0>();
      }
      __syncthreads();
      const uint32_t buf = smem_s + b * C::kSBytes;
#pragma unroll
      for (int u = 0; u < kOuCols / 32; ++u) {
        float acc[4][4] = {};
        if (has) {
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            if (ks >= steps) break;
            uint4 hi, lo;
            if (C::kRegs) {
              const uint32_t* hp = mh[C::kRegs ? ks : 0];
              const uint32_t* lp = ml[C::kRegs ? ks : 0];
              hi = make_uint4(hp[0], hp[1], hp[2], hp[3]);
              lo = make_uint4(lp[0], lp[1], lp[2], lp[3]);
            } else {
              hi = kept[(2 * ks) * 32 + lane];
              lo = kept[(2 * ks + 1) * 32 + lane];
            }
#pragma unroll
            for (int v = 0; v < 4; v += 2) {
              uint32_t f0, f1, f2, f3;
              if (FWD)
                ldmatrix_x4(buf + (32 * u + (v + (lane >> 4)) * 8 + (lane & 7)) * C::kFwdPitch + (2 * ks + ((lane >> 3) & 1)) * 16,
                            f0, f1, f2, f3);
              else
                ldmatrix_x4_trans(buf + (16 * ks + (lane & 15)) * C::kGradPitch + 64 * u + (v + (lane >> 4)) * 16, f0, f1, f2, f3);
              mma_type<TYPE>(acc[v], hi.x, hi.y, hi.z, hi.w, f0, f1);
              mma_type<TYPE>(acc[v + 1], hi.x, hi.y, hi.z, hi.w, f2, f3);
              mma_type<TYPE>(acc[v], lo.x, lo.y, lo.z, lo.w, f0, f1);
              mma_type<TYPE>(acc[v + 1], lo.x, lo.y, lo.z, lo.w, f2, f3);
            }
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int q = q0 + 32 * u;
          if (row[h] < 0 || q >= a.Q) continue;
          const uint32_t wd[4] = {was[u][h].x, was[u][h].y, was[u][h].z, was[u][h].w};
          uint32_t o[4];
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const float2 f = unpack_type<TYPE>(wd[v]);
            o[v] = has ? pack_type<TYPE>(fmaf(mul[h], acc[v][2 * h], f.x), fmaf(mul[h], acc[v][2 * h + 1], f.y)) : wd[v];
          }
          *reinterpret_cast<uint4*>(out + (int64_t)row[h] * a.out_ld + q) = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
      __syncthreads();  // before the buffer is filled again
    }
    cp_async_wait<0>();
  }
}

template <int TYPE, int KS, bool FWD>
static cudaError_t launch_out(const AdapterArgs& a, int sms, cudaStream_t st) {
  static std::atomic<bool> ready[64] = {};
  using C = OutCfg<KS>;
  const cudaError_t rc = allow_smem(adapter_out_kernel<TYPE, KS, FWD>, C::kAlloc, ready);
  if (rc != cudaSuccess) return rc;
  return launch_dependent(adapter_out_kernel<TYPE, KS, FWD>, dim3(sms * C::kCtas), dim3(kOuThreads), C::kAlloc, st, a);
}

template <int TYPE, bool FWD>
static cudaError_t launch_out(const AdapterArgs& a, int sms, cudaStream_t st) {
  if (a.R <= 16) return launch_out<TYPE, 1, FWD>(a, sms, st);
  if (a.R <= 32) return launch_out<TYPE, 2, FWD>(a, sms, st);
  if (a.R <= 64) return launch_out<TYPE, 4, FWD>(a, sms, st);
  if (a.R <= 128) return launch_out<TYPE, 8, FWD>(a, sms, st);
  return launch_out<TYPE, 16, FWD>(a, sms, st);
}

}  // namespace moe
