// The experts of a mixture-of-experts layer for a few tokens, gfx950.
//
//   h_p = act(Wg_e x_t) * (Wu_e x_t),  out_t = sum_p w_p W2_e h_p   (p: slots of t)
//
// With few tokens every product is bound by reading the selected experts' codes
// once from HBM, so the two kernels stream weight rows and keep everything else out
// of the way:
//   * 16-row tiles of codes go from global memory straight into registers, 16 bytes
//     per lane, and are converted there to the 16-bit type of the activations (one
//     instruction per two codes; MX scales are powers of two and are folded in
//     exactly).  They are the first operand of v_mfma_f32_16x16x32; up to 16 tokens
//     are its columns, so one token or sixteen cost the same weight traffic.
//   * The eight waves of a workgroup split K: together they read whole weight rows
//     at once, 16 consecutive rows of the matrix, which DRAM serves like one
//     contiguous block.  Their sums meet in LDS.
//   * A lane's 16 bytes are consecutive K, so the K order inside a matrix
//     instruction is permuted; the activations are loaded in the same order.
//   * The intermediate h is kept as two bf16 (hi + lo, 16 significant bits) and
//     costs two matrix instructions: rounding it to one bf16 would add an error of
//     the size of the output's own rounding.
//   * The second kernel writes fp32 partial rows per (token, slot) and the last
//     workgroup of a column tile adds them in slot order: no floating-point atomics,
//     the same bits on every run.
// Both kernels are persistent: every workgroup derives the experts in use and their
// slots from the ids, so the host never reads them.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "layers_device.h"

namespace fp8gemm {
namespace {

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / 64;
constexpr int kMaxPairs = kMoeMaxTokens * kMaxTopK;
constexpr int kStep = 64;            // bytes of a weight row per 16-byte load of four lane groups
constexpr int kChunk = 256;          // bytes of a weight row loaded at once: whole cache lines

// Form of the activation operand: bf16 or f16 as given; f16 split into two bf16 on
// the way (MX scales need bf16's exponent range); pairs of bf16 as the up kernel
// writes them, 8 hi then 8 lo.
enum XForm { kXBf16, kXF16, kXF16Split, kXPair };

// ---------------------------------------------------------------------------
// Experts in use and their (token, slot) pairs
// ---------------------------------------------------------------------------
struct Lists {
  int count[kMaxExperts];            // then: next free place of an expert's pairs
  int expert[kMaxExperts];           // experts in use, ascending
  int start[kMaxExperts + 1];        // their pairs: list[start[a] .. start[a+1])
  uint16_t list[kMaxPairs];          // pair = token * k + slot
  int used;
};

__device__ __forceinline__ void build_lists(Lists& l, const MoeProblem& p) {
  const int t = (int)threadIdx.x, pairs = p.T * p.k;
  for (int e = t; e < p.E; e += kThreads) l.count[e] = 0;
  __syncthreads();
  for (int i = t; i < pairs; i += kThreads) {
    const unsigned e = (unsigned)p.ids[i];
    if (e < (unsigned)p.E) atomicAdd(&l.count[e], 1);
  }
  __syncthreads();
  if (t < 64) {
    int used = 0, placed = 0;
    for (int e0 = 0; e0 < p.E; e0 += 64) {
      const int e = e0 + t;
      const int c = e < p.E ? l.count[e] : 0;
      int x = c;
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const int o = __shfl_up(x, off, 64);
        if (t >= off) x += o;
      }
      const uint64_t in_use = __ballot(c > 0);
      if (c > 0) {
        const int a = used + __popcll(in_use & ((1ull << t) - 1));
        l.expert[a] = e;
        l.start[a] = placed + x - c;
        l.count[e] = placed + x - c;
      }
      used += __popcll(in_use);
      placed += __shfl(x, 63, 64);
    }
    if (t == 0) {
      l.start[used] = placed;
      l.used = used;
    }
  }
  __syncthreads();
  // the order within an expert may differ between workgroups; a pair's values do
  // not depend on the column it takes
  for (int i = t; i < pairs; i += kThreads) {
    const unsigned e = (unsigned)p.ids[i];
    if (e < (unsigned)p.E) l.list[atomicAdd(&l.count[e], 1)] = (uint16_t)i;
  }
  __syncthreads();
}

// ---------------------------------------------------------------------------
// 16-row tiles of weight rows times columns of activations over a range of K
// ---------------------------------------------------------------------------
template <int FMT>
constexpr int kFrags = FMT == kE2M1 ? 4 : 2;         // matrix instructions per 16 bytes of codes

// Eight codes (of the 16 bytes w, fragment m) as the matrix operand; scale: a power
// of two (1 where the scale is applied to the sums).
template <int FMT, int X>
__device__ __forceinline__ u32x4 decode8(const u32x4& w, int m, float scale) {
  u32x4 r;
  if constexpr (FMT == kE2M1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      bf16x2 v;
      if (i == 0) v = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[m], scale, 0);
      if (i == 1) v = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[m], scale, 1);
      if (i == 2) v = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[m], scale, 2);
      if (i == 3) v = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[m], scale, 3);
      r[i] = __builtin_bit_cast(uint32_t, v);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t d = w[2 * m + (i >> 1)];
      if constexpr (X == kXF16) {
        const f16x2 v = (i & 1) ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(d, scale, true)
                                : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(d, scale, false);
        r[i] = __builtin_bit_cast(uint32_t, v);
      } else {
        const bf16x2 v = (i & 1) ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d, scale, true)
                                 : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d, scale, false);
        r[i] = __builtin_bit_cast(uint32_t, v);
      }
    }
  }
  return r;
}

// One lane's view of a matrix of weight rows: its row's codes (from its lane
// group's first 16 bytes on) and, with MX, its row's scale codes.
struct WeightRow {
  const uint8_t* codes;
  const uint8_t* scales;
};

template <int FMT>
struct ScaleWords {                   // the scale codes of one chunk of a row
  uint32_t w[FMT == kE2M1 ? 4 : 2];
};

template <int FMT, bool MX, int RT>
__device__ __forceinline__ void load_chunk(const WeightRow (&row)[RT], int c, int bytes, int grp,
                                           u32x4 (&w)[kChunk / kStep][RT],
                                           ScaleWords<FMT> (&sc)[RT]) {
  constexpr int kCodes = FMT == kE2M1 ? 16 : 8;      // scale codes of a chunk
  const bool full = (c + 1) * kChunk <= bytes;
#pragma unroll
  for (int s = 0; s < kChunk / kStep; ++s)
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const int off = c * kChunk + s * kStep;
      w[s][r] = u32x4{0, 0, 0, 0};
      if (full || off + grp * 16 < bytes)
        w[s][r] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(row[r].codes + off));
    }
  if constexpr (MX) {
    const int blocks = FMT == kE2M1 ? bytes / 16 : bytes / 32;
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      if (full) {
        __builtin_memcpy(sc[r].w, row[r].scales + c * kCodes, kCodes);
      } else {
#pragma unroll
        for (int i = 0; i < kCodes / 4; ++i) {
          sc[r].w[i] = 0;
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const int at = c * kCodes + 4 * i + b;
            if (at < blocks) sc[r].w[i] |= (uint32_t)row[r].scales[at] << (8 * b);
          }
        }
      }
    }
  }
}

// Scale of this lane group's block in step s of a chunk.  E4M3: a step is 64
// codes, two blocks, two lane groups each; E2M1: 128 codes, one block per group.
template <int FMT>
__device__ __forceinline__ float step_scale(const ScaleWords<FMT>& sc, int s, int grp) {
  const uint32_t code = FMT == kE2M1 ? (sc.w[s] >> (8 * grp)) & 0xffu
                                     : (sc.w[s >> 1] >> (16 * (s & 1) + 8 * (grp >> 1))) & 0xffu;
  return __uint_as_float(code << 23);
}

// acc[r][n] += rows of tile r times columns of tile n over the chunks [c0, c1).
// col[n]: this lane's column from its lane group's first element on, null: no
// column (reads nothing, counts as zero).
template <int FMT, bool MX, int X, int RT, int NT>
__device__ __forceinline__ void stream_rows(const WeightRow (&row)[RT],
                                            const uint8_t* const (&col)[NT], int bytes, int c0,
                                            int c1, int grp, f32x4 (&acc)[RT][NT]) {
  constexpr int kF = kFrags<FMT>;
  constexpr int kXFrag = X == kXPair ? 32 : 16;      // bytes of 8 activations
  constexpr int kXStep = 4 * kF * kXFrag;            // of a step: four lane groups
  u32x4 w[2][kChunk / kStep][RT];
  ScaleWords<FMT> sc[2][RT];
  if (c0 >= c1) return;
  load_chunk<FMT, MX, RT>(row, c0, bytes, grp, w[0], sc[0]);
  auto step = [&](int c, int now) __attribute__((always_inline)) {
    if (c + 1 < c1) load_chunk<FMT, MX, RT>(row, c + 1, bytes, grp, w[now ^ 1], sc[now ^ 1]);
    const bool full = (c + 1) * kChunk <= bytes;
#pragma unroll
    for (int s = 0; s < kChunk / kStep; ++s) {
      const int off = c * kChunk + s * kStep;
      const bool live = full || off + grp * 16 < bytes;
      u32x4 xv[NT][kF][kXFrag / 16];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const u32x4* from =
            reinterpret_cast<const u32x4*>(col[n] + (int64_t)(off / kStep) * kXStep);
#pragma unroll
        for (int m = 0; m < kF; ++m)
#pragma unroll
          for (int h = 0; h < kXFrag / 16; ++h) xv[n][m][h] = u32x4{0, 0, 0, 0};
        if (col[n] && live) {
#pragma unroll
          for (int m = 0; m < kF; ++m)
#pragma unroll
            for (int h = 0; h < kXFrag / 16; ++h) xv[n][m][h] = from[m * (kXFrag / 16) + h];
        }
      }
#pragma unroll
      for (int m = 0; m < kF; ++m) {
        u32x4 a[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r)
          a[r] = decode8<FMT, X>(w[now][s][r], m, MX ? step_scale<FMT>(sc[now][r], s, grp) : 1.0f);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if constexpr (X == kXF16) {
#pragma unroll
            for (int r = 0; r < RT; ++r)
              acc[r][n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                  __builtin_bit_cast(f16x8, a[r]), __builtin_bit_cast(f16x8, xv[n][m][0]),
                  acc[r][n], 0, 0, 0);
          } else {
            bf16x8 hi = __builtin_bit_cast(bf16x8, xv[n][m][0]), lo{};
            if constexpr (X == kXPair) lo = __builtin_bit_cast(bf16x8, xv[n][m][kXFrag / 16 - 1]);
            if constexpr (X == kXF16Split) {
              const f16x8 f = __builtin_bit_cast(f16x8, xv[n][m][0]);
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                __bf16 a1, a2;
                split_bf16((float)f[i], a1, a2);       // exact: 11 bits in two of 8
                hi[i] = a1;
                lo[i] = a2;
              }
            }
#pragma unroll
            for (int r = 0; r < RT; ++r) {
              acc[r][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  __builtin_bit_cast(bf16x8, a[r]), hi, acc[r][n], 0, 0, 0);
              if constexpr (X == kXPair || X == kXF16Split)
                acc[r][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    __builtin_bit_cast(bf16x8, a[r]), lo, acc[r][n], 0, 0, 0);
            }
          }
        }
      }
    }
  };
  int c = c0;
  for (; c + 1 < c1; c += 2) {
    step(c, 0);
    step(c + 1, 1);
  }
  if (c < c1) step(c, 0);
}

// Sums of the eight waves: waves store their accumulators of one column tile,
// [wave][column][row], rows padded by four against bank conflicts.
template <int RT>
struct Partials {
  float v[2][kWaves][16][16 * RT + 4];
};

template <int RT>
__device__ __forceinline__ float wave_sum(const float (&v)[kWaves][16][16 * RT + 4], int col,
                                          int row) {
  float s = 0.0f;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) s += v[w][col][row];
  return s;
}

template <int RT, int NT>
__device__ __forceinline__ void put_partials(Partials<RT>& part, int buf, int wave, int lane,
                                             const f32x4 (&acc)[RT][NT], int n) {
#pragma unroll
  for (int r = 0; r < RT; ++r)
    *reinterpret_cast<f32x4*>(&part.v[buf][wave][lane & 15][16 * r + 4 * (lane >> 4)]) = acc[r][n];
}

// Bytes of a row of `k` codes, and this wave's chunks of it.
template <int FMT>
__device__ __forceinline__ int row_bytes(int k) {
  return FMT == kE2M1 ? k / 2 : k;
}
__device__ __forceinline__ int chunk_at(int chunks, int part, int parts) {
  return (int)((int64_t)chunks * part / parts);
}

struct Workspace {
  int* arrived;                      // [column tiles of the down kernel]
  uint8_t* pair;                     // h: [T * k][I / 8][8 hi, 8 lo] bf16
  float* partial;                    // [splits][T * k][H]
  int splits;                        // of the down kernel's K
};

// ---------------------------------------------------------------------------
// h = act(Wg x) * (Wu x): a tile is 8 * RT gate rows and the same up rows
// ---------------------------------------------------------------------------
template <int FMT, int MODE, int X, int RT>
__global__ __launch_bounds__(kThreads, 2) void moe_up_kernel(MoeProblem p, Workspace ws, int tiles,
                                                             int down_tiles) {
  constexpr bool kMx = MODE == kMx32;
  constexpr int kHalf = 8 * RT;
  __shared__ Lists l;
  __shared__ Partials<RT> part;
  const int t = (int)threadIdx.x, lane = t % 64, grp = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(t / 64);
  // the down kernel's arrival counts start at zero in every call
  for (int i = (int)blockIdx.x * kThreads + t; i < down_tiles; i += (int)gridDim.x * kThreads)
    ws.arrived[i] = 0;
  build_lists(l, p);
  const int items = l.used * tiles;
  const int bytes = row_bytes<FMT>(p.H);
  const int chunks = (bytes + kChunk - 1) / kChunk;
  const int c0 = chunk_at(chunks, wave, kWaves), c1 = chunk_at(chunks, wave + 1, kWaves);
  constexpr int kXGroup = kFrags<FMT> * 16;          // bytes of a lane group's activations
  int buf = 0;
  for (int item = (int)blockIdx.x; item < items; item += (int)gridDim.x) {
    const int a = item / tiles, row0 = (item - a * tiles) * kHalf;
    const int e = __builtin_amdgcn_readfirstlane(l.expert[a]);
    const int first = __builtin_amdgcn_readfirstlane(l.start[a]);
    const int last = __builtin_amdgcn_readfirstlane(l.start[a + 1]);
    const uint8_t* w = p.w13 + (int64_t)e * p.stride13;
    WeightRow row[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const int q = 16 * r + (lane & 15);            // row of the tile: gate rows, then up rows
      const int i = row0 + (q < kHalf ? q : q - kHalf);
      const int g = (i < p.I ? i : p.I - 1) + (q < kHalf ? 0 : p.I);
      row[r].codes = w + (int64_t)g * p.ld13 + grp * 16;
      row[r].scales = kMx ? static_cast<const uint8_t*>(p.s13) +
                                ((int64_t)e * 2 * p.I + g) * (p.H / 32)
                          : nullptr;
    }
    const float* fs = static_cast<const float*>(p.s13);
    auto columns = [&](int from, auto ntag) __attribute__((always_inline)) {
      constexpr int NT = decltype(ntag)::value;
      const uint8_t* col[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int c = from + 16 * n + (lane & 15);
        col[n] = c < last ? static_cast<const uint8_t*>(p.x) +
                                (int64_t)(l.list[c] / p.k) * p.ldx * 2 + grp * kXGroup
                          : nullptr;
      }
      f32x4 acc[RT][NT];
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[r][n] = f32x4{0, 0, 0, 0};
      stream_rows<FMT, kMx, X, RT, NT>(row, col, bytes, c0, c1, grp, acc);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        put_partials<RT, NT>(part, buf, wave, lane, acc, n);
        __syncthreads();
        for (int o = t; o < 16 * kHalf; o += kThreads) {
          const int c = o / kHalf, q = o % kHalf, i = row0 + q;
          const int at = from + 16 * n + c;
          if (at < last && i < p.I) {
            float g = wave_sum<RT>(part.v[buf], c, q), u = wave_sum<RT>(part.v[buf], c, q + kHalf);
            if (MODE == kTensor) {
              g *= fs[e];
              u *= fs[e];
            }
            if (MODE == kRowwise) {
              g *= fs[(int64_t)e * 2 * p.I + i];
              u *= fs[(int64_t)e * 2 * p.I + p.I + i];
            }
            __bf16 hi, lo;
            split_bf16(layer_activate(g, p.act) * u, hi, lo);
            __bf16* to = reinterpret_cast<__bf16*>(
                ws.pair + ((int64_t)l.list[at] * p.I + (i & ~7)) * 4) + (i & 7);
            to[0] = hi;
            to[8] = lo;
          }
        }
        buf ^= 1;                     // the other buffer's readers passed the barrier above
      }
    };
    for (int from = first; from < last;) {
      const int left = last - from;
      if (left <= 16) {
        columns(from, std::integral_constant<int, 1>{});
        from += 16;
      } else if (left <= 32) {
        columns(from, std::integral_constant<int, 2>{});
        from += 32;
      } else {
        columns(from, std::integral_constant<int, 4>{});
        from += 64;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// out = sum over slots of w (W2 h): a tile is 16 * RT rows of W2, K in splits
// ---------------------------------------------------------------------------
template <int FMT, int MODE, typename OutT, int RT>
__global__ __launch_bounds__(kThreads, 2) void moe_down_kernel(MoeProblem p, Workspace ws,
                                                               int tiles) {
  constexpr bool kMx = MODE == kMx32;
  constexpr int kRows = 16 * RT;
  __shared__ Lists l;
  __shared__ Partials<RT> part;
  __shared__ int s_last;
  const int t = (int)threadIdx.x, lane = t % 64, grp = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(t / 64);
  const int pairs = p.T * p.k;
  build_lists(l, p);
  const int used = l.used;
  OutT* out = static_cast<OutT*>(p.out);
  if (used == 0) {                    // no token has an expert
    for (int64_t i = (int64_t)blockIdx.x * kThreads + t; i < (int64_t)p.T * (p.H / 4);
         i += (int64_t)gridDim.x * kThreads) {
      const float z[4] = {0, 0, 0, 0};
      store4(out + i / (p.H / 4) * p.ldo + i % (p.H / 4) * 4, z);
    }
    return;
  }
  const int items = used * ws.splits * tiles;
  const int bytes = row_bytes<FMT>(p.I);
  const int chunks = (bytes + kChunk - 1) / kChunk;
  constexpr int kXGroup = kFrags<FMT> * 32;
  const __amdgpu_buffer_rsrc_t rp =
      shared_buffer(ws.partial, (uint32_t)((int64_t)ws.splits * pairs * p.H * 4));
  const float* fs = static_cast<const float*>(p.s2);
  int buf = 0;
  for (int item = (int)blockIdx.x; item < items; item += (int)gridDim.x) {
    const int tile = item % tiles, rest = item / tiles;
    const int split = rest % ws.splits, a = rest / ws.splits;
    const int row0 = tile * kRows;
    const int part0 = split * kWaves + wave, parts = ws.splits * kWaves;
    const int c0 = chunk_at(chunks, part0, parts), c1 = chunk_at(chunks, part0 + 1, parts);
    const int e = __builtin_amdgcn_readfirstlane(l.expert[a]);
    const int first = __builtin_amdgcn_readfirstlane(l.start[a]);
    const int last = __builtin_amdgcn_readfirstlane(l.start[a + 1]);
    const uint8_t* w = p.w2 + (int64_t)e * p.stride2;
    WeightRow row[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const int q = row0 + 16 * r + (lane & 15);
      const int g = q < p.H ? q : p.H - 1;
      row[r].codes = w + (int64_t)g * p.ld2 + grp * 16;
      row[r].scales = kMx ? static_cast<const uint8_t*>(p.s2) + ((int64_t)e * p.H + g) * (p.I / 32)
                          : nullptr;
    }
    auto columns = [&](int from, auto ntag) __attribute__((always_inline)) {
      constexpr int NT = decltype(ntag)::value;
      const uint8_t* col[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int c = from + 16 * n + (lane & 15);
        col[n] = c < last ? ws.pair + (int64_t)l.list[c] * p.I * 4 + grp * kXGroup : nullptr;
      }
      f32x4 acc[RT][NT];
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[r][n] = f32x4{0, 0, 0, 0};
      stream_rows<FMT, kMx, kXPair, RT, NT>(row, col, bytes, c0, c1, grp, acc);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        put_partials<RT, NT>(part, buf, wave, lane, acc, n);
        __syncthreads();
        for (int o = t; o < 4 * kRows; o += kThreads) {
          const int c = o / (kRows / 4), q = o % (kRows / 4) * 4;
          const int at = from + 16 * n + c;
          if (at < last && row0 + q < p.H) {           // H is a multiple of 16: whole fours
            f32x4 v;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              v[i] = wave_sum<RT>(part.v[buf], c, q + i);
              if (MODE == kTensor) v[i] *= fs[e];
              if (MODE == kRowwise) v[i] *= fs[(int64_t)e * p.H + row0 + q + i];
            }
            __builtin_amdgcn_raw_buffer_store_b128(
                __builtin_bit_cast(u32x4, v), rp,
                (int)(((split * pairs + l.list[at]) * p.H + row0 + q) * 4), 0, kShared);
          }
        }
        buf ^= 1;
      }
    };
    for (int from = first; from < last;) {
      const int left = last - from;
      if (left <= 16) {
        columns(from, std::integral_constant<int, 1>{});
        from += 16;
      } else if (left <= 32) {
        columns(from, std::integral_constant<int, 2>{});
        from += 32;
      } else {
        columns(from, std::integral_constant<int, 4>{});
        from += 64;
      }
    }
    // the last of a tile's workgroups adds the slots' rows up
    __builtin_amdgcn_s_waitcnt(0);                     // this thread's rows stored
    __syncthreads();                                   // ... and every thread's
    if (t == 0)
      s_last = __hip_atomic_fetch_add(&ws.arrived[tile], 1, __ATOMIC_RELAXED,
                                      __HIP_MEMORY_SCOPE_AGENT) == used * ws.splits - 1;
    __syncthreads();
    if (s_last) {
      for (int o = t; o < p.T * (kRows / 4); o += kThreads) {
        const int tok = o / (kRows / 4), q = row0 + o % (kRows / 4) * 4;
        if (q >= p.H) continue;
        float y[4] = {0, 0, 0, 0};
        for (int j = 0; j < p.k; ++j) {
          const int i = tok * p.k + j;
          if ((unsigned)p.ids[i] >= (unsigned)p.E) continue;
          const float wt = p.weights[i];
          for (int s = 0; s < ws.splits; ++s) {
            const f32x4 v = __builtin_bit_cast(
                f32x4, __builtin_amdgcn_raw_buffer_load_b128(
                           rp, (int)(((s * pairs + i) * p.H + q) * 4), 0, kShared));
#pragma unroll
            for (int c = 0; c < 4; ++c) y[c] += wt * v[c];
          }
        }
        store4(out + (int64_t)tok * p.ldo + q, y);
      }
    }
    __syncthreads();                                   // s_last is read before it is set again
  }
}

// ---------------------------------------------------------------------------
// Launch
// ---------------------------------------------------------------------------
constexpr int kRt = 2;                 // tiles of 16 rows per workgroup step

constexpr size_t round16(size_t v) { return (v + 255) / 256 * 256; }

int down_tiles(int64_t H) { return (int)((H + 16 * kRt - 1) / (16 * kRt)); }

// K splits of the down kernel: enough work items for two workgroups per CU.
int down_splits(int64_t T, int64_t H, int64_t I, int E, int k) {
  const int64_t pairs = T * k;
  const int64_t items = down_tiles(H) * (pairs < E ? pairs : E);
  int s = 1;
  while (s < 8 && items * s < 512 && I / (2 * s) >= 1024) s *= 2;
  return s;
}

Workspace moe_layout(void* base, int64_t T, int64_t H, int64_t I, int E, int k, size_t* total) {
  Workspace ws;
  uint8_t* b = static_cast<uint8_t*>(base);
  size_t at = kSplitCounterBytes;      // the GEMMs' split-K counters: left alone
  ws.arrived = reinterpret_cast<int*>(b + at);
  at += round16((size_t)down_tiles(H) * 4);
  ws.pair = b + at;
  at += round16((size_t)T * k * I * 4);
  ws.partial = reinterpret_cast<float*>(b + at);
  ws.splits = down_splits(T, H, I, E, k);
  at += (size_t)ws.splits * T * k * H * 4;
  *total = at;
  return ws;
}

template <int FMT, int MODE, int X, typename OutT>
hipError_t launch_as(const MoeProblem& p, hipStream_t stream) {
  size_t total;
  const Workspace ws = moe_layout(p.workspace, p.T, p.H, p.I, p.E, p.k, &total);
  const int64_t pairs = (int64_t)p.T * p.k, most = pairs < p.E ? pairs : p.E;
  const int64_t slots = 2 * (int64_t)device_cu_count();
  const int up = (p.I + 8 * kRt - 1) / (8 * kRt), down = down_tiles(p.H);
  const int64_t up_items = most * up, down_items = most * down * ws.splits;
  hipLaunchKernelGGL((moe_up_kernel<FMT, MODE, X, kRt>),
                     dim3((unsigned)(up_items < slots ? up_items : slots)), dim3(kThreads), 0,
                     stream, p, ws, up, down);
  hipLaunchKernelGGL((moe_down_kernel<FMT, MODE, OutT, kRt>),
                     dim3((unsigned)(down_items < slots ? down_items : slots)), dim3(kThreads), 0,
                     stream, p, ws, down);
  return hipGetLastError();
}

template <int FMT, int MODE>
hipError_t launch_mode(const MoeProblem& p, hipStream_t stream) {
  if (p.dtype == kDtF16)
    return launch_as<FMT, MODE, MODE == kMx32 ? kXF16Split : kXF16, _Float16>(p, stream);
  return launch_as<FMT, MODE, kXBf16, __bf16>(p, stream);
}

}  // namespace

size_t moe_workspace_bytes(int64_t T, int64_t H, int64_t I, int E, int k) {
  size_t total;
  moe_layout(nullptr, T, H, I, E, k, &total);
  return total;
}

hipError_t launch_moe(const MoeProblem& p, hipStream_t stream) {
  if (p.format == kE2M1) return launch_mode<kE2M1, kMx32>(p, stream);
  if (p.mode == kTensor) return launch_mode<kE4M3, kTensor>(p, stream);
  if (p.mode == kRowwise) return launch_mode<kE4M3, kRowwise>(p, stream);
  return launch_mode<kE4M3, kMx32>(p, stream);
}

}  // namespace fp8gemm
