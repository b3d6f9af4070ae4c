// Block quantization to 8-bit floating point (E4M3 codes, one f32 scale per
// 128 elements of a row, or per 128 x 128 block of a weight).
//
// Rule, every step one f32 operation: amax over the block; scale = amax / 448
// and code = E4M3(x * (448 / amax)), rounded to nearest even. A block whose
// amax is below 2^-100 has scale 0 and codes 0 (448 / amax stays finite above
// it). An infinity or a NaN in the block becomes its scale (amax is taken on
// the bit patterns, where NaN > infinity > every number), so that each of its
// values reads back as NaN, never as a number.
//
// Rows: a warp takes 512 consecutive elements of one row, 16 a lane, so that
// a lane's codes are one 16-byte store, and eight lanes hold a block. Bytes
// bound it: the source is read once, and a row that goes to k experts is
// quantized once and stored k times.
#include "common.cuh"

#include <cuda_fp16.h>

namespace nvfp4moe {
namespace {

constexpr float kE4M3Max = 448.0f;
constexpr uint32_t kTinyBits = 0x0D800000u;   // 2^-100

// Eight consecutive elements as f32.
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* v) {
  bf16x8_to_f32(__ldg(reinterpret_cast<const uint4*>(p)), v);
}
__device__ __forceinline__ void load8(const __half* p, float* v) {
  const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void load8(const float* p, float* v) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float4 f = __ldg(reinterpret_cast<const float4*>(p) + i);
    v[4 * i] = f.x;
    v[4 * i + 1] = f.y;
    v[4 * i + 2] = f.z;
    v[4 * i + 3] = f.w;
  }
}

__device__ __forceinline__ uint32_t amax_bits16(const float (&v)[16]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  return m;
}

// Scale of a block and the factor that its elements are multiplied with.
__device__ __forceinline__ float block_scale(uint32_t amax_bits, float& inv) {
  if (amax_bits < kTinyBits) {
    inv = 0.0f;
    return 0.0f;
  }
  const float amax = __uint_as_float(amax_bits);
  inv = __fdiv_rn(kE4M3Max, amax);
  return __fdiv_rn(amax, kE4M3Max);
}

// 16 codes, element 0 in the lowest byte.
__device__ __forceinline__ uint4 encode16(const float (&v)[16], float inv) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(v[4 * i], inv), __fmul_rn(v[4 * i + 1], inv)),
                                                 __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(
        make_float2(__fmul_rn(v[4 * i + 2], inv), __fmul_rn(v[4 * i + 3], inv)), __NV_SATFINITE, __NV_E4M3);
    w[i] = lo | (hi << 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

struct RowArgs {
  const void* x;
  int64_t rows, K, ldx;
  const int32_t* f2p;   // null, or (rows, k): the rows that each source row is written to
  int k;
  int64_t n_out;        // output rows
  uint8_t* codes;
  float* sf;
  int* status;
};

// kSwiGLU: a source row holds K gate values, then K up values, and what is
// quantized is gate / (1 + exp(-gate)) * up in f32.
template <typename T, bool kSwiGLU>
__global__ void __launch_bounds__(256) quantize_rows_fp8_kernel(const RowArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t chunks = (a.K + 511) / 512;
  const int64_t item = blockIdx.x * (int64_t)(blockDim.x >> 5) + (threadIdx.x >> 5);
  const int64_t r = item / chunks;
  if (r >= a.rows) return;
  const int64_t col = (item - r * chunks) * 512 + lane * 16;
  const bool valid = col < a.K;   // K % 16 == 0: all 16 elements or none
  // lane j < k holds the row of slot j
  int64_t dst = r;
  if (a.f2p) {
    dst = -1;
    if (lane < a.k) {
      dst = a.f2p[r * a.k + lane];
      if (dst >= a.n_out) {
        if (atomicCAS(&a.status[0], 0, NVFP4MOE_ERR_INVALID) == 0) a.status[1] = 21;
        dst = -1;
      }
    }
  }
  float v[16];
  if (valid) {
    const T* p = static_cast<const T*>(a.x) + r * a.ldx + col;
    load8(p, v);
    load8(p + 8, v + 8);
    if constexpr (kSwiGLU) {
      float u[16];
      load8(p + a.K, u);
      load8(p + a.K + 8, u + 8);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = __fmul_rn(__fdiv_rn(v[i], __fadd_rn(1.0f, expf(-v[i]))), u[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = 0.0f;
  }
  uint32_t m = amax_bits16(v);
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  float inv;
  const float s = block_scale(m, inv);
  const uint4 w = encode16(v, inv);
  const int64_t nb = (a.K + 127) / 128;
  const int n = a.f2p ? a.k : 1;
  for (int j = 0; j < n; ++j) {
    const int64_t to = a.f2p ? __shfl_sync(0xFFFFFFFFu, dst, j) : r;
    if (to < 0 || !valid) continue;
    *reinterpret_cast<uint4*>(a.codes + to * a.K + col) = w;
    if ((lane & 7) == 0) a.sf[to * nb + col / 128] = s;
  }
}

// One block of 256 threads for one 128 x 128 block: thread (g, l) of 32 groups
// of eight holds 16 columns of rows g, g + 32, g + 64 and g + 96.
template <typename T>
__global__ void __launch_bounds__(256) quantize_weight_fp8_kernel(const T* __restrict__ w, int64_t N, int64_t K,
                                                                  int64_t ldw, uint8_t* __restrict__ codes,
                                                                  float* __restrict__ sf) {
  __shared__ uint32_t part[8];
  const int64_t kb = blockIdx.x, nb = blockIdx.y, e = blockIdx.z;
  const int64_t col = kb * 128 + (threadIdx.x & 7) * 16;
  float v[4][16];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t n = nb * 128 + (threadIdx.x >> 3) + 32 * i;
    if (n < N && col < K) {
      const T* p = w + (e * N + n) * ldw + col;
      load8(p, v[i]);
      load8(p + 8, v[i] + 8);
    } else {
#pragma unroll
      for (int c = 0; c < 16; ++c) v[i][c] = 0.0f;
    }
    m = max(m, amax_bits16(v[i]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, part[i]);
  float inv;
  const float s = block_scale(m, inv);
  if (threadIdx.x == 0) sf[(e * gridDim.y + nb) * gridDim.x + kb] = s;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t n = nb * 128 + (threadIdx.x >> 3) + 32 * i;
    if (n < N && col < K) *reinterpret_cast<uint4*>(codes + (e * N + n) * K + col) = encode16(v[i], inv);
  }
}

bool type_ok(int type) { return type == NVFP4MOE_BF16 || type == NVFP4MOE_F16 || type == NVFP4MOE_F32; }
int64_t type_bytes(int type) { return type == NVFP4MOE_F32 ? 4 : 2; }

template <bool kSwiGLU>
int quantize_rows(RowArgs& a, int type, void* stream) {
  NVFP4_CHECK(type_ok(type) && a.rows >= 0 && a.K >= 0 && a.K % 16 == 0 && a.rows < (1ll << 31) && a.K < (1ll << 31),
              NVFP4MOE_ERR_UNSUPPORTED);
  if (a.rows == 0 || a.K == 0) return NVFP4MOE_OK;
  NVFP4_CHECK(a.x && a.codes && a.sf, NVFP4MOE_ERR_INVALID);
  NVFP4_CHECK(a.ldx >= (kSwiGLU ? 2 : 1) * a.K && a.ldx * type_bytes(type) % 16 == 0 && aligned(a.x, 16) &&
                  aligned(a.codes, 16) && aligned(a.sf, 4),
              NVFP4MOE_ERR_INVALID);
  a.status = device_status_word();
  NVFP4_CHECK(a.status, NVFP4MOE_ERR_LAUNCH);
  const int64_t blocks = ceil_div(a.rows * ceil_div(a.K, 512), 8);
  NVFP4_CHECK(blocks < (1ll << 31), NVFP4MOE_ERR_UNSUPPORTED);
  cudaStream_t s = as_stream(stream);
  if (type == NVFP4MOE_BF16) quantize_rows_fp8_kernel<__nv_bfloat16, kSwiGLU><<<(unsigned)blocks, 256, 0, s>>>(a);
  else if (type == NVFP4MOE_F16) quantize_rows_fp8_kernel<__half, kSwiGLU><<<(unsigned)blocks, 256, 0, s>>>(a);
  else quantize_rows_fp8_kernel<float, kSwiGLU><<<(unsigned)blocks, 256, 0, s>>>(a);
  return launch_status();
}

}  // namespace
}  // namespace nvfp4moe

using namespace nvfp4moe;

extern "C" int fp8_quantize(const void* x, int type, int64_t rows, int64_t K, int64_t ldx,
                            const int32_t* flat_to_perm, int k, int64_t out_rows, uint8_t* codes, float* sf,
                            void* stream) {
  NVFP4_CHECK(out_rows >= 0 && (flat_to_perm ? k >= 1 && k <= 16 : out_rows >= rows), NVFP4MOE_ERR_UNSUPPORTED);
  RowArgs a{x, rows, K, ldx, flat_to_perm, k, out_rows, codes, sf, nullptr};
  return quantize_rows<false>(a, type, stream);
}

extern "C" int fp8_swiglu_quantize(const void* gate_up, int type, int64_t rows, int64_t I, int64_t ld,
                                   uint8_t* codes, float* sf, void* stream) {
  RowArgs a{gate_up, rows, I, ld, nullptr, 1, rows, codes, sf, nullptr};
  return quantize_rows<true>(a, type, stream);
}

extern "C" int fp8_quantize_weight(const void* w, int type, int64_t E, int64_t N, int64_t K, int64_t ldw,
                                   uint8_t* codes, float* sf, void* stream) {
  NVFP4_CHECK(type_ok(type) && E >= 0 && N >= 0 && K >= 0 && K % 16 == 0 && E <= 65535 && N <= 65535 * 128ll &&
                  K < (1ll << 31),
              NVFP4MOE_ERR_UNSUPPORTED);
  if (E == 0 || N == 0 || K == 0) return NVFP4MOE_OK;
  NVFP4_CHECK(w && codes && sf, NVFP4MOE_ERR_INVALID);
  NVFP4_CHECK(ldw >= K && ldw * type_bytes(type) % 16 == 0 && aligned(w, 16) && aligned(codes, 16) && aligned(sf, 4),
              NVFP4MOE_ERR_INVALID);
  const dim3 grid((unsigned)ceil_div(K, 128), (unsigned)ceil_div(N, 128), (unsigned)E);
  cudaStream_t s = as_stream(stream);
  if (type == NVFP4MOE_BF16)
    quantize_weight_fp8_kernel<<<grid, 256, 0, s>>>(static_cast<const __nv_bfloat16*>(w), N, K, ldw, codes, sf);
  else if (type == NVFP4MOE_F16)
    quantize_weight_fp8_kernel<<<grid, 256, 0, s>>>(static_cast<const __half*>(w), N, K, ldw, codes, sf);
  else
    quantize_weight_fp8_kernel<<<grid, 256, 0, s>>>(static_cast<const float*>(w), N, K, ldw, codes, sf);
  return launch_status();
}
