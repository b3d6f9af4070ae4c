// Block quantization to 8-bit floating point (E4M3 codes, one f32 scale per
// 128 elements of a row, or per 128 x 128 block of a weight).
//
// Rule, every step one f32 operation: amax over the block; scale = amax / 448
// and code = E4M3(x * (448 / amax)), rounded to nearest even. A block whose
// amax is below 2^-100 has scale 0 and codes 0 (448 / amax stays finite above
// it). An infinity or a NaN in the block becomes its scale (the maximum is NaN
// where either operand is), so that each of its values reads back as NaN, never
// as a number.
//
// Rows: a warp takes 512 consecutive elements of one row, 16 a lane, so that
// a lane's codes are one 16-byte store, and eight lanes hold a block. Bytes
// bound it: the source is read once, and a row that goes to k experts is
// quantized once and stored k times. Measured: 8192 x 7168 BF16 to 8 experts
// each 94 us, 6.4 TB/s of 6.76 (a plain copy's); to one place 31.7 us, 5.6
// TB/s; 8 x 4096 x 7168 BF16 weights 100 us, 7.0 TB/s. The SwiGLU form is near the
// bound of its arithmetic with 16-bit sources (16384 x 2048 BF16 29.1 us, 5.8
// TB/s; F32 44.4 us, 6.8 TB/s).
#include "common.cuh"

#include <cuda_fp16.h>

namespace nvfp4moe {
namespace {

constexpr float kE4M3Max = 448.0f;
constexpr float kTiny = 0x1p-100f;
// Warps to a block. SwiGLU, 16384 x 2048 BF16 with 1 / 2 / 4: 35.7, 29.5, 30.1 us,
// F32 44.2, 44.1, 44.6; rows, 8192 x 7168 BF16: 59.5, 31.6, 30.3.
template <bool kSwiGLU>
constexpr uint32_t kRowWarps = kSwiGLU ? 2 : 4;

// 16 consecutive elements as they lie in memory.
template <typename T>
struct Raw16 {
  uint4 w[sizeof(T)];   // 2 or 4 pieces of 16 bytes
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T); ++i) w[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  }
  // Hides the value from the compiler, which would otherwise keep the f32
  // conversions of one use (twice the registers) for the next.
  __device__ __forceinline__ void keep() {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T); ++i) asm volatile("" : "+r"(w[i].x), "+r"(w[i].y), "+r"(w[i].z), "+r"(w[i].w));
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T); ++i) w[i] = make_uint4(0u, 0u, 0u, 0u);
  }
};

__device__ __forceinline__ void to_f32(const Raw16<__nv_bfloat16>& r, float (&v)[16]) {
  bf16x8_to_f32(r.w[0], v);
  bf16x8_to_f32(r.w[1], v + 8);
}
__device__ __forceinline__ void to_f32(const Raw16<__half>& r, float (&v)[16]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t w[4] = {r.w[h].x, r.w[h].y, r.w[h].z, r.w[h].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      v[8 * h + 2 * i] = f.x;
      v[8 * h + 2 * i + 1] = f.y;
    }
  }
}
__device__ __forceinline__ void to_f32(const Raw16<float>& r, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[4 * i] = __uint_as_float(r.w[i].x);
    v[4 * i + 1] = __uint_as_float(r.w[i].y);
    v[4 * i + 2] = __uint_as_float(r.w[i].z);
    v[4 * i + 3] = __uint_as_float(r.w[i].w);
  }
}

// The larger of two numbers, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float amax16(const float (&v)[16]) {
  float m = fabsf(v[0]);
#pragma unroll
  for (int i = 1; i < 16; ++i) m = max_nan(m, fabsf(v[i]));
  return m;
}

// Scale of a block and the factor that its elements are multiplied with. A NaN
// amax is not below the bound and goes through.
__device__ __forceinline__ float block_scale(float amax, float& inv) {
  if (amax < kTiny) {
    inv = 0.0f;
    return 0.0f;
  }
  inv = __fdiv_rn(kE4M3Max, amax);
  return __fdiv_rn(amax, kE4M3Max);
}

// Two f32 operations in one instruction (a register pair each).
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint64_t pair(float a) { return pair(a, a); }
__device__ __forceinline__ void unpair(uint64_t p, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// v = silu(g) * u = g / (1 + exp(-g)) * u for two elements, within 2^-20 of it
// down to the g whose exp(-g) is an f32, below which it is 0.
//   exp(-g) = 2^t 2^d, t = -g log2(e) rounded to f32 and d the rest of the
//   product, which is up to 2^-18 and in which t would be wrong by as much:
//   2^d = 1 + d ln(2) in f32.
//   g / (1 + exp(-g)) = g/4 / ((1 + exp(-g)) / 4), since the reciprocal
//   instruction has no results below 2^-126.
// Where t overflows d is no number, and is taken as one that changes nothing.
// (16384 x 2048 BF16: 29.1 us; without d 28.8, and up to 2^-18 off; with the
// exponential and the division of CUDA's library 45.)
__device__ __forceinline__ void silu_mul2(float& v0, float& v1, float u0, float u1) {
  constexpr double kLog2e = 1.4426950408889634, kLn2 = 0.6931471805599453;
  constexpr float kHi = (float)kLog2e, kLo = (float)((kLog2e - (double)kHi) * kLn2);
  const uint64_t g = pair(v0, v1);
  const uint64_t t = mul2(g, pair(-kHi));
  const uint64_t rest = fma2(g, pair(kHi), t);                     // -d without the low part of log2(e)
  const uint64_t k = fma2(g, pair(-kLo / 4), fma2(rest, pair(-(float)kLn2 / 4), pair(0.25f)));   // 2^d / 4
  float t0, t1, k0, k1, d0, d1;
  unpair(t, t0, t1);
  unpair(k, k0, k1);
  unpair(fma2(pair(ex2(t0), ex2(t1)), pair(fminf(k0, 0.5f), fminf(k1, 0.5f)), pair(0.25f)), d0, d1);
  const uint64_t s = mul2(mul2(g, pair(0.25f)), pair(rcp(d0), rcp(d1)));
  unpair(mul2(s, pair(u0, u1)), v0, v1);
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
__global__ void __launch_bounds__(32 * kRowWarps<kSwiGLU>) quantize_rows_fp8_kernel(const RowArgs a) {
  const int lane = threadIdx.x & 31;
  // 32 bits: a 64-bit division would cost a lane as much as half its codes
  const uint32_t chunks = (uint32_t)((a.K + 511) / 512);
  const uint32_t item = blockIdx.x * kRowWarps<kSwiGLU> + (threadIdx.x >> 5);
  const int64_t r = item / chunks;
  if (r >= a.rows) return;
  const int64_t col = (int64_t)(item % chunks) * 512 + lane * 16;
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
  Raw16<T> x;
  x.zero();
  const T* p = static_cast<const T*>(a.x) + r * a.ldx + col;
  if (valid) x.load(p);
  Raw16<T> up;   // (on its way before the gate is converted: F32 44.1 us, after it 46.4)
  if constexpr (kSwiGLU) {
    up.zero();
    if (valid) up.load(p + a.K);
  }
  to_f32(x, v);
  if constexpr (kSwiGLU) {
    float u[16];
    to_f32(up, u);
#pragma unroll
    for (int i = 0; i < 16; i += 2) silu_mul2(v[i], v[i + 1], u[i], u[i + 1]);
  }
  float m = amax16(v);
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  // one division a lane: the even lanes of a block's eight make the factor, the odd ones the scale
  const bool even = (lane & 1) == 0;
  const float q = m < kTiny ? 0.0f : __fdiv_rn(even ? kE4M3Max : m, even ? m : kE4M3Max);
  const float other = __shfl_xor_sync(0xFFFFFFFFu, q, 1);
  const float inv = even ? q : other, s = even ? other : q;
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
  __shared__ float part[8];
  const int64_t kb = blockIdx.x, nb = blockIdx.y, e = blockIdx.z;
  const int64_t col = kb * 128 + (threadIdx.x & 7) * 16;
  // held as they came (32 registers for 16-bit types): more blocks on an SM
  // than with 64 f32 each
  Raw16<T> x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t n = nb * 128 + (threadIdx.x >> 3) + 32 * i;
    x[i].zero();
    if (n < N && col < K) x[i].load(w + (e * N + n) * ldw + col);
  }
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float v[16];
    to_f32(x[i], v);
    m = max_nan(m, amax16(v));
    x[i].keep();
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max_nan(m, part[i]);
  float inv;
  const float s = block_scale(m, inv);
  if (threadIdx.x == 0) sf[(e * gridDim.y + nb) * gridDim.x + kb] = s;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t n = nb * 128 + (threadIdx.x >> 3) + 32 * i;
    float v[16];
    to_f32(x[i], v);
    if (n < N && col < K) *reinterpret_cast<uint4*>(codes + (e * N + n) * K + col) = encode16(v, inv);
  }
}

bool type_ok(int type) { return type == NVFP4MOE_BF16 || type == NVFP4MOE_F16 || type == NVFP4MOE_F32; }
int64_t type_bytes(int type) { return type == NVFP4MOE_F32 ? 4 : 2; }

template <bool kSwiGLU>
int quantize_rows(RowArgs& a, int type, void* stream) {
  NVFP4_CHECK(type_ok(type) && a.rows >= 0 && a.K >= 0 && a.K % 16 == 0 && a.rows < (1ll << 31) && a.K < (1ll << 31),
              NVFP4MOE_ERR_UNSUPPORTED);
  if (a.rows == 0 || a.K == 0) return NVFP4MOE_OK;
  NVFP4_CHECK(a.x && (a.n_out == 0 || (a.codes && a.sf)), NVFP4MOE_ERR_INVALID);
  NVFP4_CHECK(a.ldx >= (kSwiGLU ? 2 : 1) * a.K && a.ldx * type_bytes(type) % 16 == 0 && aligned(a.x, 16) &&
                  aligned(a.codes, 16) && aligned(a.sf, 4),
              NVFP4MOE_ERR_INVALID);
  a.status = device_status_word();
  NVFP4_CHECK(a.status, NVFP4MOE_ERR_LAUNCH);
  const int64_t items = a.rows * ceil_div(a.K, 512), blocks = ceil_div(items, kRowWarps<kSwiGLU>);
  NVFP4_CHECK(items < (1ll << 32) - 8, NVFP4MOE_ERR_UNSUPPORTED);
  const unsigned threads = 32 * kRowWarps<kSwiGLU>;
  cudaStream_t s = as_stream(stream);
  if (type == NVFP4MOE_BF16) quantize_rows_fp8_kernel<__nv_bfloat16, kSwiGLU><<<(unsigned)blocks, threads, 0, s>>>(a);
  else if (type == NVFP4MOE_F16) quantize_rows_fp8_kernel<__half, kSwiGLU><<<(unsigned)blocks, threads, 0, s>>>(a);
  else quantize_rows_fp8_kernel<float, kSwiGLU><<<(unsigned)blocks, threads, 0, s>>>(a);
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
