// Low-rank adapters of many requests beside a shared projection, gfx950.
//
//   v_p = x_m A_g^T                       (shrink: rank values per row)
//   out_m = act(base_m + s_g v_p B_g^T)   (expand)        m = order[p], p in group g
//
// Rows come sorted by adapter (order, offsets), so a tile of up to 16 * NT rows has one
// adapter and both products run on v_mfma_f32_16x16x32 with the adapter's rows as the
// first operand and the rows of x or v as its columns:
//   * shrink: the waves of a workgroup split K (and workgroups too where rows are few);
//     the fp32 sums go to the workspace by position, one slice per split, and are added
//     in slice order by the expand kernel: no atomics, the same bits on every run.
//   * expand: v keeps 16 bits or more as two 16-bit operands (bf16 hi + lo; for f16
//     rows scaled by a power of two first, so that v cannot leave f16's range), so the
//     output is rounded once.  The columns of the matrix operand are dealt so that a
//     lane ends with 16 consecutive outputs of one row.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "layers_device.h"

namespace fp8gemm {
namespace {

// ---------------------------------------------------------------------------
// Tiles of rows
// ---------------------------------------------------------------------------
struct RowTile {
  int group;            // `groups`: rows without an adapter
  int first, last;      // positions in `order`
};

// Tile `index` of the groups' rows cut into tiles of `rows` positions; the rows of
// no group are a last group where with_rest.  False: there are fewer tiles.  Offsets
// are clamped into [0, M].  Every thread of the workgroup takes part.
template <int THREADS>
__device__ __forceinline__ bool find_tile(const int32_t* offsets, int groups, int M, int rows,
                                          bool with_rest, int index, RowTile& tile) {
  __shared__ int scratch[THREADS / 64];
  __shared__ RowTile found;
  const int t = (int)threadIdx.x, lane = t % 64, wave = t / 64;
  const int n = groups + (with_rest ? 1 : 0);
  const int per = (n + THREADS - 1) / THREADS;
  auto range = [&](int g, int& a, int& b) {
    a = offsets[g];
    b = g < groups ? offsets[g + 1] : M;
    a = a < 0 ? 0 : (a > M ? M : a);
    b = b < a ? a : (b > M ? M : b);
  };
  int mine = 0;
  for (int g = t * per; g < n && g < (t + 1) * per; ++g) {
    int a, b;
    range(g, a, b);
    mine += (b - a + rows - 1) / rows;
  }
  int x = mine;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int o = __shfl_up(x, off, 64);
    if (lane >= off) x += o;
  }
  if (lane == 63) scratch[wave] = x;
  if (t == 0) found.group = -1;
  __syncthreads();
  int before = x - mine;
  for (int w = 0; w < wave; ++w) before += scratch[w];
  if (index >= before && index < before + mine) {
    int at = before;
    for (int g = t * per; g < n && g < (t + 1) * per; ++g) {
      int a, b;
      range(g, a, b);
      const int c = (b - a + rows - 1) / rows;
      if (index < at + c) {
        found.group = g;
        found.first = a + (index - at) * rows;
        found.last = found.first + rows < b ? found.first + rows : b;
        break;
      }
      at += c;
    }
  }
  __syncthreads();
  tile.group = __builtin_amdgcn_readfirstlane(found.group);
  tile.first = __builtin_amdgcn_readfirstlane(found.first);
  tile.last = __builtin_amdgcn_readfirstlane(found.last);
  return tile.group >= 0;
}

template <typename T>
__device__ __forceinline__ f32x4 mfma16(const u32x4& a, const u32x4& b, f32x4 c) {
  if constexpr (std::is_same<T, _Float16>::value)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// ---------------------------------------------------------------------------
// Shrink
// ---------------------------------------------------------------------------
constexpr int kShrinkThreads = 512;
constexpr int kShrinkWaves = kShrinkThreads / 64;
constexpr int kShrinkChunk = 128;      // elements of K loaded at once: 256 bytes of a row

// RT tiles of 16 adapter rows (from r0 on) by NT tiles of 16 rows of x.
template <typename T, int RT, int NT>
__global__ __launch_bounds__(kShrinkThreads, 2) void lora_shrink_kernel(LoraProblem p, float* v,
                                                                       int splits, int rblocks) {
  __shared__ float part[kShrinkWaves][16][16 * RT + 4];
  const int t = (int)threadIdx.x, lane = t % 64, grp = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(t / 64);
  int id = (int)blockIdx.x;
  const int split = id % splits;
  id /= splits;
  const int r0 = id % rblocks * 16 * RT;
  RowTile tile;
  if (!find_tile<kShrinkThreads>(p.offsets, p.groups, p.M, 16 * NT, false, id / rblocks, tile))
    return;
  const T* a = static_cast<const T*>(p.a) + (int64_t)tile.group * p.stride_a;
  const T* arow[RT];
  const T* xrow[NT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int q = r0 + 16 * r + (lane & 15);
    arow[r] = q < p.rank ? a + (int64_t)q * p.lda + grp * 8 : nullptr;
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int pos = tile.first + 16 * n + (lane & 15);
    const int m = pos < tile.last ? p.order[pos] : -1;
    xrow[n] = (unsigned)m < (unsigned)p.M ? static_cast<const T*>(p.x) + (int64_t)m * p.ldx + grp * 8
                                          : nullptr;
  }
  f32x4 acc[RT][NT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[r][n] = f32x4{0, 0, 0, 0};
  const int chunks = (p.K + kShrinkChunk - 1) / kShrinkChunk;
  const int parts = splits * kShrinkWaves, at = split * kShrinkWaves + wave;
  const int c0 = (int)((int64_t)chunks * at / parts), c1 = (int)((int64_t)chunks * (at + 1) / parts);
  for (int c = c0; c < c1; ++c) {
    u32x4 aw[4][RT], xw[4][NT];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int k = c * kShrinkChunk + s * 32;
      const bool live = k + grp * 8 < p.K;             // K is a multiple of 8
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        aw[s][r] = u32x4{0, 0, 0, 0};
        if (live && arow[r]) aw[s][r] = *reinterpret_cast<const u32x4*>(arow[r] + k);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        xw[s][n] = u32x4{0, 0, 0, 0};
        if (live && xrow[n]) xw[s][n] = *reinterpret_cast<const u32x4*>(xrow[n] + k);
      }
    }
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[r][n] = mfma16<T>(aw[s][r], xw[s][n], acc[r][n]);
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    if (n > 0) __syncthreads();
#pragma unroll
    for (int r = 0; r < RT; ++r)
      *reinterpret_cast<f32x4*>(&part[wave][lane & 15][16 * r + 4 * grp]) = acc[r][n];
    __syncthreads();
    for (int o = t; o < 16 * 16 * RT; o += kShrinkThreads) {
      const int c = o / (16 * RT), q = o % (16 * RT), pos = tile.first + 16 * n + c;
      if (pos < tile.last && r0 + q < p.rank) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kShrinkWaves; ++w) s += part[w][c][q];
        v[((int64_t)split * p.M + pos) * p.rank + r0 + q] = s;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Expand
// ---------------------------------------------------------------------------
constexpr int kExpandThreads = 256;
constexpr int kExpandCols = 64 * (kExpandThreads / 64);   // output columns of a workgroup

// MT tiles of 16 rows by 64 columns per wave; KS steps of 32 cover the rank.
template <typename T, int KS, int MT>
__global__ __launch_bounds__(kExpandThreads, 2) void lora_expand_kernel(LoraProblem p,
                                                                       const float* v, int splits,
                                                                       int nblocks) {
  const int t = (int)threadIdx.x, lane = t % 64, grp = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(t / 64);
  const int id = (int)blockIdx.x;
  RowTile tile;
  if (!find_tile<kExpandThreads>(p.offsets, p.groups, p.M, 16 * MT, true, id / nblocks, tile))
    return;
  const int n0 = id % nblocks * kExpandCols + wave * 64;
  if (n0 >= p.N) return;
  const bool adapted = tile.group < p.groups;

  // B's rows for output column n0 + 16 g' + 4 t + i sit in row 4 g' + i of tile t,
  // so that lane group g' ends with columns 16 g' .. 16 g' + 15
  u32x4 b[KS][4];
  if (adapted) {
    const T* bg = static_cast<const T*>(p.b) + (int64_t)tile.group * p.stride_b;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int n = n0 + 16 * ((lane & 15) >> 2) + 4 * c + (lane & 3);
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const int k = 32 * s + 8 * grp;
        b[s][c] = u32x4{0, 0, 0, 0};
        if (n < p.N && k < p.rank)
          b[s][c] = *reinterpret_cast<const u32x4*>(bg + (int64_t)n * p.ldb + k);
      }
    }
  }
  const float scale = adapted && p.scales ? p.scales[tile.group] : 1.0f;

  for (int m = 0; m < MT; ++m) {
    const int pos = tile.first + 16 * m + (lane & 15);
    if (tile.first + 16 * m >= tile.last) break;
    f32x4 acc[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[c] = f32x4{0, 0, 0, 0};
    float back = scale;
    if (adapted) {
      float f[KS][8];
#pragma unroll
      for (int s = 0; s < KS; ++s) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[s][i] = 0.0f;
        const int k = 32 * s + 8 * grp;
        if (pos < tile.last && k < p.rank)
          for (int q = 0; q < splits; ++q) {
            const f32x4* from = reinterpret_cast<const f32x4*>(
                v + ((int64_t)q * p.M + pos) * p.rank + k);
            const f32x4 lo4 = from[0], hi4 = from[1];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              f[s][i] += lo4[i];
              f[s][4 + i] += hi4[i];
            }
          }
      }
      if constexpr (std::is_same<T, _Float16>::value) {
        // |v| scaled into [1, 2): 22 bits in two f16, none out of range
        float mx = 0.0f;
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int i = 0; i < 8; ++i) mx = fmaxf(mx, fabsf(f[s][i]));
        mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
        mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
        const int ex = mx > 0.0f ? (int)(__float_as_uint(mx) >> 23) - 127 : 0;
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int i = 0; i < 8; ++i) f[s][i] = ldexpf(f[s][i], -ex);
        back = ldexpf(scale, ex);
      }
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        T hi[8], lo[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          hi[i] = (T)f[s][i];
          lo[i] = (T)(f[s][i] - (float)hi[i]);
        }
        u32x4 vh, vl;
        __builtin_memcpy(&vh, hi, 16);
        __builtin_memcpy(&vl, lo, 16);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          acc[c] = mfma16<T>(b[s][c], vh, acc[c]);
          acc[c] = mfma16<T>(b[s][c], vl, acc[c]);
        }
      }
    }
    const int row = pos < tile.last ? p.order[pos] : -1;
    const int n = n0 + 16 * grp;
    if ((unsigned)row >= (unsigned)p.M || n >= p.N) continue;
    const T* base = static_cast<const T*>(p.base) + (int64_t)row * p.ldbase + n;
    T* out = static_cast<T*>(p.out) + (int64_t)row * p.ldo + n;
    if (n + 16 <= p.N) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        T w[8];
        const u32x4 in = reinterpret_cast<const u32x4*>(base)[h];
        __builtin_memcpy(w, &in, 16);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          w[i] = to_out<T>(layer_activate((float)w[i] + back * acc[2 * h + (i >> 2)][i & 3], p.act));
        u32x4 o;
        __builtin_memcpy(&o, w, 16);
        reinterpret_cast<u32x4*>(out)[h] = o;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (n + i < p.N)
          out[i] = to_out<T>(layer_activate((float)base[i] + back * acc[i >> 2][i & 3], p.act));
    }
  }
}

// ---------------------------------------------------------------------------
// Launch
// ---------------------------------------------------------------------------
// Tiles that M rows in at most `groups` runs are cut into, at most.
int64_t most_tiles(int64_t M, int64_t groups, int rows) {
  return M / rows + (groups < M ? groups : M);
}

// K slices of the shrink kernel: where rows are few, enough workgroups for every CU.
int shrink_splits(int64_t M, int64_t K, int groups) {
  int s = 1;
  while (s < 8 && most_tiles(M, groups, 32) * s < 256 && K / (2 * s) >= 1024) s *= 2;
  return s;
}

template <typename T, int RT>
hipError_t launch_shrink(const LoraProblem& p, float* v, int splits, hipStream_t stream) {
  const int rblocks = (p.rank + 16 * RT - 1) / (16 * RT);
  const int64_t grid = most_tiles(p.M, p.groups, 32) * rblocks * splits;
  hipLaunchKernelGGL((lora_shrink_kernel<T, RT, 2>), dim3((unsigned)grid), dim3(kShrinkThreads), 0,
                     stream, p, v, splits, rblocks);
  return hipGetLastError();
}

template <typename T, int KS>
hipError_t launch_expand(const LoraProblem& p, const float* v, int splits, hipStream_t stream) {
  const int nblocks = (p.N + kExpandCols - 1) / kExpandCols;
  const int64_t grid = (most_tiles(p.M, p.groups + 1, 32)) * nblocks;
  hipLaunchKernelGGL((lora_expand_kernel<T, KS, 2>), dim3((unsigned)grid), dim3(kExpandThreads), 0,
                     stream, p, v, splits, nblocks);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_as(const LoraProblem& p, hipStream_t stream) {
  float* v = reinterpret_cast<float*>(static_cast<uint8_t*>(p.workspace) + kSplitCounterBytes);
  const int splits = shrink_splits(p.M, p.K, p.groups);
  hipError_t e = p.rank <= 16   ? launch_shrink<T, 1>(p, v, splits, stream)
                 : p.rank <= 32 ? launch_shrink<T, 2>(p, v, splits, stream)
                                : launch_shrink<T, 4>(p, v, splits, stream);
  if (e != hipSuccess) return e;
  if (p.rank <= 32) return launch_expand<T, 1>(p, v, splits, stream);
  if (p.rank <= 64) return launch_expand<T, 2>(p, v, splits, stream);
  return launch_expand<T, 4>(p, v, splits, stream);
}

}  // namespace

size_t lora_workspace_bytes(int64_t M, int64_t K, int rank, int groups) {
  return (size_t)kSplitCounterBytes +
         (size_t)shrink_splits(M, K, groups) * (size_t)M * (size_t)rank * sizeof(float);
}

hipError_t launch_lora(const LoraProblem& p, hipStream_t stream) {
  return p.dtype == kDtF16 ? launch_as<_Float16>(p, stream) : launch_as<__bf16>(p, stream);
}

}  // namespace fp8gemm
