// mx.cu -- microscaled 4-bit matrices (include/zipnn.h): quantisation and reading back.
//
// Both are one pass over the data with a few operations a value, so HBM bounds them: BF16 to
// MXFP4 moves 2 + 0.5 + 1/32 bytes a value each way.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "zipnn.h"
#include "common.cuh"
#include "launch.h"
#include "mx.cuh"

namespace zipnn {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t kMaxPartials = ZIPNN_MX_WORKSPACE_BYTES / 4;
constexpr int kChunk = 16;  // values of one thread: 8 bytes of codes

// Threads of a block cover `rows_per` rows x `chunk_cols` (a power of two) chunks.
struct Cover {
  uint32_t log_cols;   // log2 of chunk_cols
  uint32_t col_tiles;  // blocks of chunks along a row
  uint64_t tiles;
};

Cover cover(uint64_t rows, uint64_t chunks) {
  Cover c;
  c.log_cols = 0;
  while ((1ull << c.log_cols) < chunks && (1 << c.log_cols) < kThreads) c.log_cols++;
  c.col_tiles = (uint32_t)mx_div_up(chunks, 1ull << c.log_cols);
  c.tiles = mx_div_up(rows, (uint64_t)kThreads >> c.log_cols) * c.col_tiles;
  return c;
}

__device__ __forceinline__ void place(const Cover& c, uint64_t tile, uint64_t& row, uint32_t& chunk) {
  const uint64_t rt = tile / c.col_tiles;
  const uint32_t ct = (uint32_t)(tile - rt * c.col_tiles);
  row = rt * (kThreads >> c.log_cols) + (threadIdx.x >> c.log_cols);
  chunk = (ct << c.log_cols) + (threadIdx.x & ((1u << c.log_cols) - 1));
}

struct Matrix {
  const uint8_t* base;
  const uint8_t* end;  // past the last row's last value
  uint64_t rows, stride_bytes;
  uint32_t cols;
};

template <int TYPE>
__device__ __forceinline__ float value_at(const uint8_t* p) {
  if constexpr (TYPE == kValFP32) return *reinterpret_cast<const float*>(p);
  if constexpr (TYPE == kValBF16) return __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(p) << 16);
  return __half2float(*reinterpret_cast<const __half*>(p));
}

// Values 16 * chunk .. 16 * chunk + 15 of a row, zeros past its end. Whole 16-byte vectors
// around them are loaded where they lie inside the matrix, whatever the row's own alignment
// (a row of odd length starts anywhere), and shifted into place; the matrix's first and last
// bytes are read value by value.
template <int TYPE>
__device__ __forceinline__ void load_chunk(const Matrix& m, uint64_t row, uint32_t chunk, float (&v)[kChunk]) {
  constexpr int B = (int)mx_value_bytes(TYPE), W = kChunk * B / 4;
  const uint32_t first = chunk * kChunk;
  if (row >= m.rows || first >= m.cols) {
#pragma unroll
    for (int i = 0; i < kChunk; i++) v[i] = 0.f;
    return;
  }
  const uint8_t* p = m.base + row * m.stride_bytes + (uint64_t)first * B;
  const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15);
  const uint8_t* a = p - off;
  const uint32_t left = m.cols - first;
  if (a >= m.base && a + W * 4 + (off ? 16 : 0) <= m.end) {
    uint32_t w[W + 4];
#pragma unroll
    for (int i = 0; i < W / 4; i++) {
      const uint4 t = __ldg(reinterpret_cast<const uint4*>(a) + i);
      w[4 * i] = t.x, w[4 * i + 1] = t.y, w[4 * i + 2] = t.z, w[4 * i + 3] = t.w;
    }
    if (off) {
      const uint4 t = __ldg(reinterpret_cast<const uint4*>(a) + W / 4);
      w[W] = t.x, w[W + 1] = t.y, w[W + 2] = t.z, w[W + 3] = t.w;
      if (off & 8) {
#pragma unroll
        for (int i = 0; i < W + 2; i++) w[i] = w[i + 2];
      }
      if (off & 4) {
#pragma unroll
        for (int i = 0; i < W + 1; i++) w[i] = w[i + 1];
      }
      if (off & 2) {
#pragma unroll
        for (int i = 0; i < W; i++) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
      }
    }
#pragma unroll
    for (int i = 0; i < kChunk; i++) {
      if constexpr (TYPE == kValFP32) {
        v[i] = __uint_as_float(w[i]);
      } else if constexpr (TYPE == kValBF16) {
        v[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
      } else {
        v[i] = __half2float(__ushort_as_half((unsigned short)(w[i / 2] >> (i & 1 ? 16 : 0))));
      }
    }
    if (left < kChunk) {
#pragma unroll
      for (int i = 0; i < kChunk; i++) v[i] = (uint32_t)i < left ? v[i] : 0.f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kChunk; i++) v[i] = (uint32_t)i < left ? value_at<TYPE>(p + i * B) : 0.f;
  }
}

// Two FP32 quotients to a byte of two E2M1 codes (the first in the low nibble), four such
// bytes: the type's own rounding, ties to even, saturating.
__device__ __forceinline__ uint32_t to_e2m1(const float* q) {
  uint32_t r;
  asm("{\n .reg .b8 b0, b1, b2, b3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
      " mov.b32 %0, {b0, b1, b2, b3};\n}\n"
      : "=r"(r)
      : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
  return r;
}

__device__ __forceinline__ uint32_t to_e4m3(float x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
  return r & 0xFF;
}
__device__ __forceinline__ float from_e4m3(uint32_t b) {
  uint32_t h2;
  const uint16_t in = (uint16_t)b;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(in));
  return __half2float(__ushort_as_half((unsigned short)h2));
}

// The E4M3 code nearest to amax / (6 g). The FP32 quotient is off by less than 4 of its last
// steps; where a border between two codes is nearer than that, or the quotient leaves the
// range where the borders have at most 4 bits, it is taken again in 64 bits and rounded to
// odd in FP32 (23 bits and a sticky one hold every border apart).
__device__ __forceinline__ uint32_t nv_scale(float amax, float g, float inv6g) {
  float t = amax * inv6g;
  const uint32_t low = (__float_as_uint(t) + 8) & 0x7FFFF;
  if (low < 16 || !(t >= 0.0156250f && t <= 1e30f)) {
    const double want = (double)amax / (6.0 * (double)g);
    t = __double2float_rz(want);
    if ((double)t != want) t = __uint_as_float(__float_as_uint(t) | 1u);
  }
  return to_e4m3(t);
}

// The codes of a block's values for the scale s g. q = x * (1 / (s g)) is off by less than 4
// of its last steps; a quotient within that of a border between two E2M1 values (its low 21
// fraction bits are then near 0) sends the thread to the comparison of |x| with the seven
// borders times s g, which is exact: border * s has 7 bits, and its product with g rounded
// up or down separates |x| >= border from |x| > border.
__device__ __forceinline__ void nv_codes(const float (&v)[kChunk], float s, float g, uint32_t (&codes)[2]) {
  const float unit = s * g;
  if (s == 0.f) {
    float z[kChunk];
#pragma unroll
    for (int i = 0; i < kChunk; i++) z[i] = copysignf(0.f, v[i]);
    codes[0] = to_e2m1(z), codes[1] = to_e2m1(z + 8);
    return;
  }
  const float inv = __frcp_rn(unit);
  float q[kChunk];
  uint32_t near = 0xFFFFFFFFu;
#pragma unroll
  for (int i = 0; i < kChunk; i++) {
    q[i] = v[i] * inv;
    near = min(near, (__float_as_uint(q[i]) + 4) & 0x1FFFFF);
  }
  codes[0] = to_e2m1(q), codes[1] = to_e2m1(q + 8);
  if (near < 8 || !(unit >= 1e-30f && unit <= 1e30f)) {
    const float border[7] = {0.25f, 0.75f, 1.25f, 1.75f, 2.5f, 3.5f, 5.f};
    float t[7];
#pragma unroll
    for (int k = 0; k < 7; k++) t[k] = k & 1 ? __fmul_ru(border[k] * s, g) : __fmul_rd(border[k] * s, g);
    codes[0] = codes[1] = 0;
#pragma unroll
    for (int i = 0; i < kChunk; i++) {
      const float x = fabsf(v[i]);
      uint32_t c = 0;
#pragma unroll
      for (int k = 0; k < 7; k++) c += k & 1 ? x >= t[k] : x > t[k];
      c |= __float_as_uint(v[i]) >> 31 << 3;
      codes[i / 8] |= c << (4 * (i % 8));
    }
  }
}

__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* smem) {
  v = __reduce_max_sync(0xFFFFFFFFu, v);
  if (threadIdx.x % 32 == 0) smem[threadIdx.x / 32] = v;
  __syncthreads();
  v = smem[threadIdx.x % (kThreads / 32)];
  return __reduce_max_sync(0xFFFFFFFFu, v);
}

// The largest finite magnitude of each block's share of the matrix, to partial[blockIdx.x].
template <int TYPE>
__global__ void __launch_bounds__(kThreads) k_mx_amax(Matrix m, Cover c, uint32_t* partial) {
  __shared__ uint32_t smem[kThreads / 32];
  uint32_t top = 0;
  for (uint64_t t = blockIdx.x; t < c.tiles; t += gridDim.x) {
    uint64_t row;
    uint32_t chunk;
    place(c, t, row, chunk);
    float v[kChunk];
    load_chunk<TYPE>(m, row, chunk, v);
#pragma unroll
    for (int i = 0; i < kChunk; i++) {
      const uint32_t u = __float_as_uint(v[i]) & 0x7FFFFFFF;
      top = max(top, u < 0x7F800000 ? u : 0);
    }
  }
  top = block_max(top, smem);
  if (threadIdx.x == 0) partial[blockIdx.x] = top;
}

// One thread quantises 16 values: half an MXFP4 block (its other half in the lane beside it)
// or an NVFP4 block, with one load of its values, 8 bytes of codes stored, and the scales of
// four blocks joined by shuffles into one word of their tile.
template <int FMT, int TYPE>
__global__ void __launch_bounds__(kThreads) k_mx_quantize(Matrix m, Cover c, float* global_scale,
                                                          const uint32_t* partial, uint32_t n_partial, uint8_t* codes,
                                                          uint8_t* scales, uint64_t row_bytes, uint64_t col_tiles) {
  float g = 1.f, inv6g = 0.f;
  if constexpr (FMT == kNvFp4) {
    if (n_partial) {
      __shared__ uint32_t smem[kThreads / 32];
      uint32_t top = 0;
      for (uint32_t i = threadIdx.x; i < n_partial; i += kThreads) top = max(top, partial[i]);
      top = block_max(top, smem);
      g = __fdiv_rn(__uint_as_float(top), 2688.f);
      if (g == 0.f) g = 1.f;
      if (blockIdx.x == 0 && threadIdx.x == 0) *global_scale = g;
    } else {
      g = *global_scale;
    }
    inv6g = __frcp_rn(6.f * g);
  }
  for (uint64_t t = blockIdx.x; t < c.tiles; t += gridDim.x) {
    uint64_t row;
    uint32_t chunk;
    place(c, t, row, chunk);
    float v[kChunk];
    load_chunk<TYPE>(m, row, chunk, v);
    uint32_t top = 0;  // as integers, so that a NaN is above every number
#pragma unroll
    for (int i = 0; i < kChunk; i++) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFF);
    uint32_t out[2] = {0, 0}, word;
    if constexpr (FMT == kMxFp4) {
      top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
      uint32_t byte = 255;
      if (top < 0x7F800000) {
        // the exponent field less 2: floor(log2(amax)) - 2 + 127, and 0 below the range
        byte = (uint32_t)max((int)(top >> 23) - 2, 0);
        const float inv = __uint_as_float((254 - byte) << 23);  // 2^(127 - byte), a normal number
        float q[kChunk];
#pragma unroll
        for (int i = 0; i < kChunk; i++) q[i] = v[i] * inv;  // exact where it matters: above 2^-126
        out[0] = to_e2m1(q), out[1] = to_e2m1(q + 8);
      }
      word = byte << (8 * (chunk / 2 % 4));
      word |= __shfl_xor_sync(0xFFFFFFFFu, word, 2);
      word |= __shfl_xor_sync(0xFFFFFFFFu, word, 4);
    } else {
      uint32_t byte = 127;
      if (top < 0x7F800000) {
        byte = nv_scale(__uint_as_float(top), g, inv6g);
        nv_codes(v, from_e4m3(byte), g, out);
      }
      word = byte << (8 * (chunk % 4));
      word |= __shfl_xor_sync(0xFFFFFFFFu, word, 1);
      word |= __shfl_xor_sync(0xFFFFFFFFu, word, 2);
    }
    if (row < m.rows && (uint64_t)chunk * 8 < row_bytes)
      *reinterpret_cast<uint2*>(codes + row * row_bytes + (uint64_t)chunk * 8) = make_uint2(out[0], out[1]);
    constexpr uint32_t kPer = FMT == kMxFp4 ? 8 : 4;  // chunks of four blocks
    const uint64_t tile = chunk / kPer;
    if (chunk % kPer == 0 && tile < col_tiles && row < mx_div_up(m.rows, 128) * 128)
      *reinterpret_cast<uint32_t*>(scales + (row / 128 * col_tiles + tile) * kMxTileBytes +
                                   mx_in_tile((uint32_t)(row % 128), 0)) = word;
  }
}

template <int FMT>
__device__ __forceinline__ float scale_of(uint32_t b) {
  if constexpr (FMT == kMxFp4)  // 2^(b - 127): b = 0 is below the normal numbers
    return __uint_as_float(b == 255 ? 0x7FFFFFFFu : b ? b << 23 : 0x400000u);
  return from_e4m3(b);
}

// One thread writes one aligned 16-byte vector of the output (8 or 4 values), wherever rows
// of odd length start: it is the codes, 4 bits each, that are shifted into place. The vector
// lies in at most two blocks.
template <int FMT, int TYPE>
__global__ void __launch_bounds__(kThreads) k_mx_dequantize(const uint8_t* codes, const uint8_t* scales,
                                                            const float* global_scale, uint64_t rows, uint32_t cols,
                                                            uint8_t* out, uint64_t stride_bytes, Cover c,
                                                            uint64_t row_bytes, uint64_t col_tiles) {
  constexpr int B = (int)mx_value_bytes(TYPE), V = 16 / B;
  constexpr uint32_t kBlk = mx_block(FMT);
  const float g = FMT == kNvFp4 ? *global_scale : 1.f;
  for (uint64_t t = blockIdx.x; t < c.tiles; t += gridDim.x) {
    uint64_t row;
    uint32_t vec;
    place(c, t, row, vec);
    if (row >= rows) continue;
    uint8_t* o = out + row * stride_bytes;
    const int64_t e0 = (int64_t)vec * V - (int64_t)((reinterpret_cast<uintptr_t>(o) & 15) / B);
    if (e0 >= (int64_t)cols) continue;
    const int64_t lo = e0 < 0 ? 0 : e0, hi = e0 + V < (int64_t)cols ? e0 + V : (int64_t)cols;  // values lo .. hi - 1
    const uint32_t* w = reinterpret_cast<const uint32_t*>(codes + row * row_bytes);
    const int64_t w0 = e0 >> 3;
    const uint32_t sh = 4 * (uint32_t)(e0 & 7);
    uint32_t bits = w0 >= 0 ? __ldg(w + w0) : 0u;
    if (sh + 4 * V > 32) bits = __funnelshift_r(bits, (uint64_t)(w0 + 1) * 4 < row_bytes ? __ldg(w + w0 + 1) : 0u, sh);
    else bits >>= sh;
    const uint32_t b0 = (uint32_t)lo / kBlk, b1 = (uint32_t)(hi - 1) / kBlk;
    const uint8_t* st = scales + row / 128 * col_tiles * kMxTileBytes;
    const uint32_t r = (uint32_t)(row % 128);
    const float s0 = scale_of<FMT>(__ldg(st + (uint64_t)(b0 / 4) * kMxTileBytes + mx_in_tile(r, b0)));
    const float s1 = b1 == b0 ? s0 : scale_of<FMT>(__ldg(st + (uint64_t)(b1 / 4) * kMxTileBytes + mx_in_tile(r, b1)));
    const int cut = (int)((int64_t)(b0 + 1) * kBlk - e0);  // values from here on are of the second block
    float v[V];
#pragma unroll
    for (int i = 0; i < V / 2; i++) {
      uint32_t h2;
      asm("{\n .reg .b8 b, z1, z2, z3;\n mov.b32 {b, z1, z2, z3}, %1;\n cvt.rn.f16x2.e2m1x2 %0, b;\n}\n"
          : "=r"(h2)
          : "r"(bits >> (8 * i)));
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
      v[2 * i] = f.x * (2 * i < cut ? s0 : s1);
      v[2 * i + 1] = f.y * (2 * i + 1 < cut ? s0 : s1);
    }
    if constexpr (FMT == kNvFp4) {
#pragma unroll
      for (int i = 0; i < V; i++) v[i] *= g;
    }
    uint32_t p[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      if constexpr (TYPE == kValFP32) {
        p[i] = __float_as_uint(v[i]);
      } else if constexpr (TYPE == kValBF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        p[i] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
        p[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    uint8_t* at = o + e0 * B;
    if (lo == e0 && hi == e0 + V) {
      *reinterpret_cast<uint4*>(at) = make_uint4(p[0], p[1], p[2], p[3]);
    } else {
#pragma unroll
      for (int i = 0; i < V; i++) {
        if (e0 + i < lo || e0 + i >= hi) continue;
        if constexpr (TYPE == kValFP32) reinterpret_cast<uint32_t*>(at)[i] = p[i];
        else reinterpret_cast<uint16_t*>(at)[i] = (uint16_t)(p[i / 2] >> (16 * (i % 2)));
      }
    }
  }
}

uint32_t grid_of(uint64_t tiles, uint32_t most) { return (uint32_t)(tiles < most ? tiles : most); }
constexpr uint32_t kGrid = 148 * 8;  // every thread of the device at 256 a block

template <int TYPE>
cudaError_t launch_quantize(int fmt, const Matrix& m, float* global_scale, bool find, uint8_t* codes, uint8_t* scales,
                            uint32_t* partial, cudaStream_t st) {
  const uint64_t col_tiles = mx_col_tiles(fmt, m.cols), chunks = col_tiles * (4 * mx_block(fmt) / kChunk);
  uint32_t n_partial = 0;
  if (fmt == kNvFp4 && find) {
    const Cover ca = cover(m.rows, mx_div_up(m.cols, kChunk));
    n_partial = grid_of(ca.tiles, kMaxPartials);
    TimedLaunch t(kIdMxAmax, st);
    k_mx_amax<TYPE><<<n_partial, kThreads, 0, st>>>(m, ca, partial);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  const Cover c = cover(mx_div_up(m.rows, 128) * 128, chunks);
  const uint64_t rb = mx_row_bytes(m.cols);
  TimedLaunch t(kIdMxQuantize, st);
  if (fmt == kMxFp4)
    k_mx_quantize<kMxFp4, TYPE><<<grid_of(c.tiles, kGrid), kThreads, 0, st>>>(m, c, nullptr, nullptr, 0, codes, scales, rb, col_tiles);
  else
    k_mx_quantize<kNvFp4, TYPE><<<grid_of(c.tiles, kGrid), kThreads, 0, st>>>(m, c, global_scale, partial, n_partial, codes, scales, rb, col_tiles);
  return cudaGetLastError();
}

template <int FMT, int TYPE>
cudaError_t launch_dequantize(const uint8_t* codes, const uint8_t* scales, const float* g, uint64_t rows, uint32_t cols,
                              uint8_t* out, uint64_t stride_bytes, cudaStream_t st) {
  constexpr uint32_t V = 16 / mx_value_bytes(TYPE);
  // a row that starts off a 16-byte boundary has one vector more
  const bool even = reinterpret_cast<uintptr_t>(out) % 16 == 0 && stride_bytes % 16 == 0;
  const Cover c = cover(rows, even ? mx_div_up(cols, V) : (uint64_t)cols / V + 2);
  TimedLaunch t(kIdMxDequantize, st);
  k_mx_dequantize<FMT, TYPE><<<grid_of(c.tiles, kGrid), kThreads, 0, st>>>(codes, scales, g, rows, cols, out, stride_bytes, c,
                                                                           mx_row_bytes(cols), mx_col_tiles(FMT, cols));
  return cudaGetLastError();
}

inline bool off16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) != 0; }
inline zipnn_status cuda_status(cudaError_t e) { return e == cudaSuccess ? ZIPNN_OK : ZIPNN_ERR_CUDA; }

}  // namespace
}  // namespace zipnn

using namespace zipnn;

extern "C" {

size_t zipnn_mx_row_bytes(uint64_t cols) { return cols && cols <= kMxMaxCols ? (size_t)mx_row_bytes(cols) : 0; }

size_t zipnn_mx_scale_bytes(zipnn_mx_format format, uint64_t rows, uint64_t cols) {
  if (!mx_valid(format, rows, cols)) return 0;
  return (size_t)(mx_div_up(rows, 128) * mx_col_tiles(format, cols) * kMxTileBytes);
}

zipnn_status zipnn_mx_quantize(zipnn_mx_format format, zipnn_value_type type, const void* x, uint64_t rows,
                               uint64_t cols, uint64_t row_stride, float* global_scale, int find_global, void* codes,
                               void* scales, void* ws, size_t ws_bytes, zipnn_stream_t stream) {
  if (!mx_valid(format, rows, cols) || !mx_valid_type(type) || !x || !codes || !scales || off16(codes) || off16(scales))
    return ZIPNN_ERR_INVALID_ARG;
  const uint32_t B = mx_value_bytes(type);
  if (reinterpret_cast<uintptr_t>(x) % B || row_stride < cols || row_stride > kMxMaxCols) return ZIPNN_ERR_INVALID_ARG;
  const bool find = format == ZIPNN_NVFP4 && find_global;
  if (format == ZIPNN_NVFP4 && (!global_scale || reinterpret_cast<uintptr_t>(global_scale) % 4)) return ZIPNN_ERR_INVALID_ARG;
  if (find && (!ws || off16(ws))) return ZIPNN_ERR_INVALID_ARG;
  if (find && ws_bytes < ZIPNN_MX_WORKSPACE_BYTES) return ZIPNN_ERR_OUT_TOO_SMALL;
  if (!device_ok()) return ZIPNN_ERR_UNSUPPORTED;
  Matrix m;
  m.base = static_cast<const uint8_t*>(x);
  m.rows = rows;
  m.cols = (uint32_t)cols;
  m.stride_bytes = row_stride * B;
  m.end = m.base + (rows - 1) * m.stride_bytes + cols * B;
  uint8_t *c = static_cast<uint8_t*>(codes), *s = static_cast<uint8_t*>(scales);
  uint32_t* p = static_cast<uint32_t*>(ws);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (type == ZIPNN_VALUE_BF16) return cuda_status(launch_quantize<kValBF16>(format, m, global_scale, find, c, s, p, st));
  if (type == ZIPNN_VALUE_FP32) return cuda_status(launch_quantize<kValFP32>(format, m, global_scale, find, c, s, p, st));
  return cuda_status(launch_quantize<kValFP16>(format, m, global_scale, find, c, s, p, st));
}

zipnn_status zipnn_mx_dequantize(zipnn_mx_format format, zipnn_value_type type, const void* codes, const void* scales,
                                 const float* global_scale, uint64_t rows, uint64_t cols, void* out,
                                 uint64_t row_stride, zipnn_stream_t stream) {
  if (!mx_valid(format, rows, cols) || !mx_valid_type(type) || !codes || !scales || !out || off16(codes) || off16(scales))
    return ZIPNN_ERR_INVALID_ARG;
  const uint32_t B = mx_value_bytes(type);
  if (reinterpret_cast<uintptr_t>(out) % B || row_stride < cols || row_stride > kMxMaxCols) return ZIPNN_ERR_INVALID_ARG;
  if (format == ZIPNN_NVFP4 && (!global_scale || reinterpret_cast<uintptr_t>(global_scale) % 4)) return ZIPNN_ERR_INVALID_ARG;
  if (!device_ok()) return ZIPNN_ERR_UNSUPPORTED;
  const uint8_t *c = static_cast<const uint8_t*>(codes), *s = static_cast<const uint8_t*>(scales);
  uint8_t* o = static_cast<uint8_t*>(out);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const uint32_t n = (uint32_t)cols;
#define ZIPNN_MX_CASE(F, T) \
  if (format == F && type == T) return cuda_status(launch_dequantize<F, T>(c, s, global_scale, rows, n, o, row_stride * B, st));
  ZIPNN_MX_CASE(kMxFp4, kValBF16)
  ZIPNN_MX_CASE(kMxFp4, kValFP32)
  ZIPNN_MX_CASE(kMxFp4, kValFP16)
  ZIPNN_MX_CASE(kNvFp4, kValBF16)
  ZIPNN_MX_CASE(kNvFp4, kValFP32)
  ZIPNN_MX_CASE(kNvFp4, kValFP16)
#undef ZIPNN_MX_CASE
  return ZIPNN_ERR_INVALID_ARG;
}

}  // extern "C"
