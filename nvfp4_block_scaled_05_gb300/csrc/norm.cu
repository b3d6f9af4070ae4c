// RMS norm of rows with the residual's addition: h = x + r rounded to its type,
//   y = h * inv * gamma,  inv = 1 / sqrt(sum(h^2) / K + eps),
// y in 16 or 32 bits, as E4M3 codes with one scale per 128 elements (the rule of
// fp8_quantize.cu, on y in f32), or both; and the gradients
//   g = dy * gamma,  dx = inv * (g - h * inv^2 * sum(g * h) / K) + dh,
//   d_gamma = sum over rows of dy * h * inv.
// Squares, sums, inv, g and d_gamma are f32, every result is rounded once. Bytes
// bound it: every operand is read once.
//
// Three forms. Rows whose runs of eight elements start on 16-byte boundaries: a row
// a block, in registers, for the shortest way from load to store. Many such rows,
// where 16-bit ones are wide or in the backward pass: persistent blocks with the
// next rows on their way into shared memory. Rows at any alignment: the aligned
// pieces of 16 bytes that lie within a row, and the elements before and after them
// by themselves.
#include "fp8_rows.cuh"

#include <type_traits>

namespace nvfp4moe {
namespace {

constexpr int64_t kMaxWidth = 16384;     // two padded f32 rows in shared memory
constexpr int kRun = 8;                  // neighbouring elements of a thread
constexpr int64_t kSharedOfBlock = 227 * 1024;

struct NormArgs {
  const void *x, *r, *dy, *dh;   // forward: x and r (or null); backward: dy, and dh (or null)
  const float* gamma;
  void *h, *y;                   // forward: results (or null); backward: h is read, y is dx
  uint8_t* codes;
  float *sf, *parts;             // parts: d_gamma's partial sums, (parts, K)
  int64_t rows, ldx, ldr, ldh, ldy, lddy, lddh;
  int K;
  float eps, inv_K;
  int tpr, groups;               // threads to a row, rows at a time in a block
  int stages;                    // rows that a block has in shared memory or on their way
  uint64_t wait_limit_ns;
  int* status;
  int test_stall;                // test hook: the first wait is for a barrier that nothing arrives on
};

__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ void from_float(__nv_bfloat16& d, float v) { d = __float2bfloat16_rn(v); }
__device__ __forceinline__ void from_float(__half& d, float v) { d = __float2half_rn(v); }
__device__ __forceinline__ void from_float(float& d, float v) { d = v; }

template <typename T>
__device__ __forceinline__ float2 to_float2(uint32_t w) {
  if constexpr (std::is_same<T, __half>::value) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  else return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));   // BF16
}
template <typename T>
__device__ __forceinline__ uint32_t from_float2(float a, float b) {
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}

// Eight neighbouring elements, computed with as four pairs (an instruction takes two
// f32: many rows of 7168 BF16 to codes are bound by issue, 69% of it with one each).
// (Not the read-only path: they may lie where the kernel writes, each read and
// written by its owner only.)
template <typename T>
struct Run {
  uint4 w[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) w[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(p)[i] = w[i];
  }
  // as four pairs of f32
  __device__ __forceinline__ void get(uint64_t (&f)[kRun / 2]) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        f[2 * i] = pair(__uint_as_float(w[i].x), __uint_as_float(w[i].y));
        f[2 * i + 1] = pair(__uint_as_float(w[i].z), __uint_as_float(w[i].w));
      }
    } else {
      const uint32_t v[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 q = to_float2<T>(v[i]);
        f[i] = pair(q.x, q.y);
      }
    }
  }
  __device__ __forceinline__ void set(const uint64_t (&f)[kRun / 2]) {
    float v[kRun];
#pragma unroll
    for (int i = 0; i < 4; ++i) unpair(f[i], v[2 * i], v[2 * i + 1]);
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        w[i] = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]),
                          __float_as_uint(v[4 * i + 3]));
    } else {
      w[0] = make_uint4(from_float2<T>(v[0], v[1]), from_float2<T>(v[2], v[3]), from_float2<T>(v[4], v[5]),
                        from_float2<T>(v[6], v[7]));
    }
  }
  // hides the value, whose f32 form (twice the registers) would otherwise be kept for the next use
  __device__ __forceinline__ void keep() {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i)
      asm volatile("" : "+r"(w[i].x), "+r"(w[i].y), "+r"(w[i].z), "+r"(w[i].w));
  }
};
__device__ __forceinline__ void load8(const float* p, uint64_t (&f)[kRun / 2]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  f[0] = pair(a.x, a.y), f[1] = pair(a.z, a.w), f[2] = pair(b.x, b.y), f[3] = pair(b.z, b.w);
}

__device__ __forceinline__ float inverse(const NormArgs& a, float squares) {
  return rsqrtf(fmaf(squares, a.inv_K, a.eps));
}

// h of x and r.
template <typename T>
__device__ __forceinline__ void add_residual(Run<T>& h, const Run<T>& r) {
  uint64_t f[kRun / 2], g[kRun / 2];
  h.get(f);
  r.get(g);
#pragma unroll
  for (int i = 0; i < kRun / 2; ++i) f[i] = add2(f[i], g[i]);
  h.set(f);
}
template <typename T>
__device__ __forceinline__ uint64_t squares(const Run<T>& h, uint64_t s) {
  uint64_t f[kRun / 2];
  h.get(f);
#pragma unroll
  for (int i = 0; i < kRun / 2; ++i) s = fma2(f[i], f[i], s);
  return s;
}
__device__ __forceinline__ float both(uint64_t s) {
  float a, b;
  unpair(s, a, b);
  return a + b;
}

// y of eight elements from column `col` on, stored and quantized; sixteen lanes
// (all called) hold a block of 128. `in`: the elements exist (gamma is 0 else).
template <typename T>
__device__ __forceinline__ void put_result(const NormArgs& a, int64_t row, int col, bool in, const Run<T>& h, float inv,
                                           const uint64_t (&gamma)[kRun / 2]) {
  uint64_t f[kRun / 2];
  h.get(f);
  const uint64_t inv2 = pair(inv);
#pragma unroll
  for (int i = 0; i < kRun / 2; ++i) f[i] = mul2(mul2(f[i], inv2), gamma[i]);
  if (a.y && in) {
    Run<T> y;
    y.set(f);
    y.store(static_cast<T*>(a.y) + row * a.ldy + col);
  }
  if (a.codes) {
    float v[kRun];
#pragma unroll
    for (int i = 0; i < kRun / 2; ++i) unpair(f[i], v[2 * i], v[2 * i + 1]);
    float m = fabsf(v[0]);
#pragma unroll
    for (int i = 1; i < kRun; ++i) m = max_nan(m, fabsf(v[i]));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    // one division a lane: the even lanes make the factor, the odd ones the scale
    const bool even = (threadIdx.x & 1) == 0;
    const float mine = m < kTiny ? 0.0f : __fdiv_rn(even ? kE4M3Max : m, even ? m : kE4M3Max);
    const float other = __shfl_xor_sync(0xFFFFFFFFu, mine, 1);
    if (in) {
      *reinterpret_cast<uint2*>(a.codes + row * a.K + col) = encode8(f, even ? mine : other);
      if ((threadIdx.x & 15) == 0) a.sf[row * ((a.K + 127) / 128) + col / 128] = other;
    }
  }
}

// dx of eight elements, and their share of d_gamma.
template <typename T>
__device__ __forceinline__ void put_gradient(const NormArgs& a, int64_t row, int col, const Run<T>& h, Run<T>& d,
                                             const Run<T>& e, float inv, float c, const uint64_t (&gamma)[kRun / 2],
                                             uint64_t (&acc)[kRun / 2]) {
  uint64_t f[kRun / 2], g[kRun / 2];
  h.get(f);
  d.get(g);
  const uint64_t inv2 = pair(inv), c2 = pair(-c);
#pragma unroll
  for (int i = 0; i < kRun / 2; ++i) {
    acc[i] = fma2(g[i], mul2(f[i], inv2), acc[i]);
    g[i] = mul2(inv2, fma2(f[i], c2, mul2(g[i], gamma[i])));
  }
  if (a.dh) {
    e.get(f);
#pragma unroll
    for (int i = 0; i < kRun / 2; ++i) g[i] = add2(g[i], f[i]);
  }
  d.set(g);
  d.store(static_cast<T*>(a.y) + row * a.ldy + col);
}

// Sums over the lanes of a row (a power of two up to 32).
template <int N>
__device__ __forceinline__ void lane_sums(float (&s)[N], int lanes) {
  for (int o = lanes >> 1; o > 0; o >>= 1) {
#pragma unroll
    for (int n = 0; n < N; ++n) s[n] += __shfl_xor_sync(0xFFFFFFFFu, s[n], o);
  }
}

// ------------------------------------------------------------------ a row a block

// P runs to a thread, one row (or, of few threads each, several) to a block.
template <typename T, int P>
__global__ void __launch_bounds__(512, 1) rms_norm_kernel(const NormArgs a) {
  __shared__ float part[16];
  const int t = threadIdx.x % a.tpr, K = a.K;
  const int64_t row = (int64_t)blockIdx.x * a.groups + threadIdx.x / a.tpr;
  const bool live = row < a.rows;
  Run<T> h[P], r[P];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int col = (p * a.tpr + t) * kRun;
    h[p].zero();
    if (live && col < K) {
      h[p].load(static_cast<const T*>(a.x) + row * a.ldx + col);
      if (a.r) r[p].load(static_cast<const T*>(a.r) + row * a.ldr + col);
    }
  }
  uint64_t gamma[P][kRun / 2];   // on their way with the row
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int col = (p * a.tpr + t) * kRun;
    if (col < K) load8(a.gamma + col, gamma[p]);
    else gamma[p][0] = gamma[p][1] = gamma[p][2] = gamma[p][3] = 0;
  }
  uint64_t sq = 0;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int col = (p * a.tpr + t) * kRun;
    if (a.r && live && col < K) {
      add_residual(h[p], r[p]);
      h[p].store(static_cast<T*>(a.h) + row * a.ldh + col);
    }
    sq = squares(h[p], sq);
    h[p].keep();
  }
  float s[1] = {both(sq)};
  lane_sums(s, a.tpr < 32 ? a.tpr : 32);
  if (a.tpr > 32) {
    const int warps = a.tpr >> 5, first = (threadIdx.x >> 5) / warps * warps;
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s[0];
    __syncthreads();
    s[0] = 0.0f;
    for (int i = 0; i < warps; ++i) s[0] += part[first + i];
  }
  const float inv = inverse(a, s[0]);
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int col = (p * a.tpr + t) * kRun;
    put_result(a, row, col, live && col < K, h[p], inv, gamma[p]);
  }
}

// ------------------------------------------------------------------ many rows
//
// A persistent block of several groups of threads; its rows go to the groups in
// turn, and the next `stages` rows' operands are on their way into shared memory
// (bulk copies: 100 KB and more on their way to an SM, which rows in registers
// cannot have). A group synchronizes by itself, so that one's sums and divisions
// run under the others' loads and stores; its barrier frees the row's place for the
// next copy. (8192 rows of 7168, BF16 with a residual: to codes 70.8 us, 5.8 TB/s of
// 6.8; to BF16 83 and backward 82, 5.7 TB/s; issue and DRAM bound them.)

constexpr int kMaxStages = 64;
// Forward, 16-bit rows of 12 KB and more. A block of registers reads gamma anew for
// each row, 4 bytes an element beside 2 to 8 of the operands, which is what narrow and
// F32 rows do not feel. us, a row a block and copied ahead, to codes with a
// residual: 9728 rows of 7168 BF16 105.7 and 85.7, 1216 14.6 and 14.0, 608 8.4 and
// 9.8; 2432 of 16384 67.0 and 55.0; 9728 of 4096 52.9 and 54.0, of 2048 27.1 and
// 26.3, of 512 7.4 and 15.9; 4864 of 7168 F32 70.4 and 77.5.
// Backward, 16-bit rows up to 14336 wide and F32 up to 8192 (a row's threads are one
// group at most; wider rows take the form for any alignment: 2048 of 16384 BF16 97.2).
// us with dh, that form and copied ahead, for 304, 608, 1216 and 2432 rows: 1024 BF16
// 6.5 and 9.6, 8.3 and 10.1, 10.5 and 10.6, 14.5 and 13.6; 7168 BF16 12.0 and 12.5,
// 16.3 and 15.1, 25.4 and 20.6, 46.7 and 31.0; 14336 BF16 16.3 and 18.6, 24.1 and
// 25.7, 56.9 and 36.5, 101 and 58; 7168 F32 11.9 and 13.4, 17.4 and 18.1, 50.3 and
// 29.3, 91 and 50. Eight rows an SM is where narrow rows break even; wide ones do
// between two and six (912 of 7168 F32 36.8 and 24.8).
constexpr int64_t kWideRow = 6144;
constexpr int64_t kRowsOfSM = 8;

struct RingTail {
  uint64_t full[kMaxStages], never;
  int fills[kMaxStages];
  float part[2][2 * 32];
  int gave_up;
};
int64_t ring_bytes(int64_t K, int64_t es, int operands, int stages) {
  return 4 * K + stages * operands * K * es + (int64_t)sizeof(RingTail) + 16;
}

template <typename T, int N>
struct RowRing {
  uint8_t* stage0;
  RingTail* tail;
  const T* src[N];
  int64_t ld[N];
  int64_t row;       // at hand
  int n, at;         // operands in use; the row's stage
  uint32_t phase;
  int group, t, warp;

  __device__ __forceinline__ RowRing(const NormArgs& a, uint8_t* smem, int operands) {
    n = operands;
    stage0 = smem + 4 * (int64_t)a.K;
    tail = reinterpret_cast<RingTail*>(stage0 + (int64_t)a.stages * n * a.K * sizeof(T));
    group = threadIdx.x / a.tpr;
    t = threadIdx.x - group * a.tpr;
    warp = t >> 5;
    at = group;
    phase = 0;
    row = blockIdx.x + (int64_t)group * gridDim.x;
    float* gamma = reinterpret_cast<float*>(smem);
    for (int c = 4 * threadIdx.x; c < a.K; c += 4 * blockDim.x)
      *reinterpret_cast<float4*>(gamma + c) = __ldg(reinterpret_cast<const float4*>(a.gamma + c));
    if (threadIdx.x == 0) {
      tail->gave_up = 0;
      for (int i = 0; i < a.stages; ++i) {
        mbar_init(smem_addr(&tail->full[i]), 1);
        tail->fills[i] = 0;
      }
      mbar_init(smem_addr(&tail->never), 1);
      fence_mbar_init();
    }
    __syncthreads();
  }
  // by one thread
  __device__ __forceinline__ void issue(const NormArgs& a, int s, int64_t from) {
    if (from >= a.rows) return;
    const uint32_t bar = smem_addr(&tail->full[s]), bytes = (uint32_t)a.K * (uint32_t)sizeof(T);
    tail->fills[s] += 1;
    mbar_arrive_expect_tx(bar, bytes * n);
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < n)
        bulk_load(smem_addr(stage0 + ((int64_t)s * n + i) * bytes), src[i] + from * ld[i], bytes, bar,
                  l2_policy_evict_first());
  }
  __device__ __forceinline__ void start(const NormArgs& a) {
    if (threadIdx.x == 0)
      for (int i = 0; i < a.stages; ++i) issue(a, i, blockIdx.x + (int64_t)i * gridDim.x);
    __syncthreads();   // (fills[] passes to the groups)
  }
  __device__ __forceinline__ const T* operand(const NormArgs& a, int i) const {
    return reinterpret_cast<const T*>(stage0) + ((int64_t)at * n + i) * a.K;
  }
  // The row at hand has landed. (Its place is the group's own, see launch_rows: a
  // group that could reach another's place would take that one's earlier phase, not
  // over yet, for the later one's end.)
  __device__ __forceinline__ bool wait(const NormArgs& a, int site) {
    return wait_bounded(smem_addr(a.test_stall ? &tail->never : &tail->full[at]), phase, &tail->gave_up, a.wait_limit_ns,
                        a.status, site);
  }
  // Sums over the group; false in all of it if one is not ok. All of it has read the
  // row's operands.
  template <int M>
  __device__ __forceinline__ bool sums(const NormArgs& a, float (&s)[M], bool ok, int turn) {
    lane_sums(s, 32);
    const int warps = a.tpr >> 5;
    if (warps == 1) return __all_sync(0xFFFFFFFFu, ok);
    float* part = tail->part[turn] + group * warps;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int m = 0; m < M; ++m) part[32 * m + warp] = s[m];
    }
    uint32_t failed;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\tbar.red.or.pred q, %1, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(failed)
        : "r"(group + 1), "r"(a.tpr), "r"(ok ? 0u : 1u)
        : "memory");
    if (failed) return false;
#pragma unroll
    for (int m = 0; m < M; ++m) {
      s[m] = 0.0f;
      for (int i = 0; i < warps; ++i) s[m] += part[32 * m + i];
    }
    return true;
  }
  // the row's place takes the next copy; on to the group's next row's
  __device__ __forceinline__ void release(const NormArgs& a) {
    __syncwarp();
    if (t == 0) issue(a, at, row + (int64_t)a.stages * gridDim.x);
    at += a.groups;
    if (at >= a.stages) {   // (a multiple of the groups)
      at -= a.stages;
      phase ^= 1;
    }
  }
  // after the last row: a block that gave up waits for its copies in flight
  __device__ __forceinline__ void drain(const NormArgs& a) {
    __syncthreads();
    if (tail->gave_up && threadIdx.x == 0)
      for (int i = 0; i < a.stages; ++i)
        if (tail->fills[i]) drain_wait(smem_addr(&tail->full[i]), (tail->fills[i] - 1) & 1);
  }
};

template <typename T, int P, int kThreads>
__global__ void __launch_bounds__(kThreads, 1) rms_norm_rows_kernel(const NormArgs a) {
  extern __shared__ __align__(128) uint8_t norm_smem[];
  const int K = a.K;
  const float* gamma = reinterpret_cast<const float*>(norm_smem);
  RowRing<T, 2> ring(a, norm_smem, a.r ? 2 : 1);
  ring.src[0] = static_cast<const T*>(a.x), ring.ld[0] = a.ldx;
  ring.src[1] = static_cast<const T*>(a.r), ring.ld[1] = a.ldr;
  ring.start(a);
  int turn = 0;
  for (; ring.row < a.rows; ring.row += (int64_t)a.groups * gridDim.x, turn ^= 1) {
    const bool ok = ring.wait(a, 61);
    Run<T> h[P];
    uint64_t sq = 0;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int col = (p * a.tpr + ring.t) * kRun;
      h[p].zero();
      if (col < K) {
        h[p].load(ring.operand(a, 0) + col);
        if (a.r) {
          Run<T> r;
          r.load(ring.operand(a, 1) + col);
          add_residual(h[p], r);
        }
      }
      sq = squares(h[p], sq);
      h[p].keep();
    }
    float s[1] = {both(sq)};
    if (!ring.sums(a, s, ok, turn)) break;
    ring.release(a);
    const float inv = inverse(a, s[0]);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int col = (p * a.tpr + ring.t) * kRun;
      const bool in = col < K;
      uint64_t w[kRun / 2] = {};
      if (in) {
        load8(gamma + col, w);
        if (a.r) h[p].store(static_cast<T*>(a.h) + ring.row * a.ldh + col);
      }
      put_result(a, ring.row, col, in, h[p], inv, w);
    }
  }
  ring.drain(a);
}

template <typename T, int P, int kThreads>
__global__ void __launch_bounds__(kThreads, 1) rms_norm_backward_rows_kernel(const NormArgs a) {
  extern __shared__ __align__(128) uint8_t norm_smem[];
  const int K = a.K;
  const float* gamma = reinterpret_cast<const float*>(norm_smem);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  RowRing<T, 3> ring(a, norm_smem, a.dh ? 3 : 2);
  ring.src[0] = static_cast<const T*>(a.h), ring.ld[0] = a.ldh;
  ring.src[1] = static_cast<const T*>(a.dy), ring.ld[1] = a.lddy;
  ring.src[2] = static_cast<const T*>(a.dh), ring.ld[2] = a.lddh;
  ring.start(a);
  uint64_t acc[P][kRun / 2] = {};
  int turn = 0;
  for (; ring.row < a.rows; ring.row += (int64_t)a.groups * gridDim.x, turn ^= 1) {
    const bool ok = ring.wait(a, 62);
    Run<T> h[P], d[P], e[P];
    uint64_t s0 = 0, s1 = 0;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int col = (p * a.tpr + ring.t) * kRun;
      if (col >= K) continue;
      uint64_t f[kRun / 2], g[kRun / 2], w[kRun / 2];
      h[p].load(ring.operand(a, 0) + col);
      d[p].load(ring.operand(a, 1) + col);
      if (a.dh) e[p].load(ring.operand(a, 2) + col);
      load8(gamma + col, w);
      h[p].get(f);
      d[p].get(g);
#pragma unroll
      for (int i = 0; i < kRun / 2; ++i) {
        s0 = fma2(f[i], f[i], s0);
        s1 = fma2(mul2(g[i], w[i]), f[i], s1);
      }
      h[p].keep();
      d[p].keep();
    }
    float s[2] = {both(s0), both(s1)};
    if (!ring.sums(a, s, ok, turn)) break;
    ring.release(a);
    const float inv = inverse(a, s[0]), c = inv * inv * (s[1] * a.inv_K);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int col = (p * a.tpr + ring.t) * kRun;
      if (col >= K) continue;
      uint64_t w[kRun / 2];
      load8(gamma + col, w);
      put_gradient(a, ring.row, col, h[p], d[p], e[p], inv, c, w, acc[p]);
    }
  }
  ring.drain(a);
  // the groups' shares of d_gamma, added up in order where the rows were
  __syncthreads();
  float* shares = reinterpret_cast<float*>(ring.stage0);
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int col = (p * a.tpr + ring.t) * kRun;
    if (col < K) {
#pragma unroll
      for (int i = 0; i < kRun / 2; ++i)
        unpair(acc[p][i], shares[(int64_t)ring.group * K + col + 2 * i],
               shares[(int64_t)ring.group * K + col + 2 * i + 1]);
    }
  }
  __syncthreads();
  for (int col = threadIdx.x; col < K; col += blockDim.x) {
    float v = 0.0f;
    for (int g = 0; g < a.groups; ++g) v += shares[(int64_t)g * K + col];
    a.parts[(int64_t)blockIdx.x * K + col] = v;
  }
}

// ------------------------------------------------------------------ any alignment
//
// Rows of odd widths start anywhere, but a row of one operand mostly where that of
// another does, so that their 16-byte pieces hold the same columns. A persistent
// block takes a row at a time: its pieces, then the few elements before the first
// and after the last one (all elements, where the operands' rows do not start
// alike). Which columns a thread has differs from row to row, so that gamma and
// d_gamma's sums are in shared memory, with a word of padding a piece against bank
// conflicts, and so is the row between the two passes where there is room.
// (4096 x 7167 BF16 with a residual 81 us, backward 80, bound by instructions; element
// by element 145 and 177, aligned rows of 7000 in the other forms 44 and 45.)

template <typename T>
constexpr int kPiece = 16 / (int)sizeof(T);
template <typename T>
__host__ __device__ constexpr int padded(int c) {
  return c + c / kPiece<T>;
}
template <typename T>
__host__ __device__ constexpr int gamma_bytes(int K) {
  return (padded<T>(K) * 4 + 15) / 16 * 16;
}
// The pieces, then the elements outside them (where the rows start alike, fewer than
// two pieces; else all, from the beginning).
template <typename T>
__host__ __device__ constexpr int row_bytes(int K) {
  return (K / kPiece<T> + 2) * 16;
}

template <typename T, bool kBackward>
__global__ void __launch_bounds__(512, 2) rms_norm_any_kernel(const NormArgs a) {
  extern __shared__ __align__(128) uint8_t norm_smem[];
  __shared__ float part[2][32];
  constexpr int V = kPiece<T>;
  const int K = a.K, tid = threadIdx.x, step = blockDim.x, warps = step >> 5;
  float* gamma = reinterpret_cast<float*>(norm_smem);
  float* acc = reinterpret_cast<float*>(norm_smem + gamma_bytes<T>(K));                               // backward
  T* hs = reinterpret_cast<T*>(norm_smem + gamma_bytes<T>(K) * (kBackward ? 2 : 1));
  T* ds = reinterpret_cast<T*>(reinterpret_cast<uint8_t*>(hs) + row_bytes<T>(K));                   // backward
  const bool keep = a.stages != 0;
  if (kBackward) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (int c = tid; c < K; c += step) {
    gamma[padded<T>(c)] = __ldg(a.gamma + c);
    if (kBackward) acc[padded<T>(c)] = 0.0f;
  }
  __syncthreads();
  struct alignas(16) Piece {
    T v[V];
  };
  int turn = 0;
  bool before = true;   // the last row's `alike`
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    const T* x = kBackward ? static_cast<const T*>(a.h) + row * a.ldh : static_cast<const T*>(a.x) + row * a.ldx;
    const T* r = kBackward ? static_cast<const T*>(a.dy) + row * a.lddy
                 : a.r     ? static_cast<const T*>(a.r) + row * a.ldr
                           : nullptr;
    T* h = !kBackward && r ? static_cast<T*>(a.h) + row * a.ldh : nullptr;
    const T* e = kBackward && a.dh ? static_cast<const T*>(a.dh) + row * a.lddh : nullptr;
    T* y = static_cast<T*>(a.y) + row * a.ldy;
    auto start = [](const void* p) { return (int)(reinterpret_cast<uintptr_t>(p) & 15); };
    const int s0 = start(x);
    const bool alike = (!r || start(r) == s0) && (!h || start(h) == s0) && (!e || start(e) == s0) && start(y) == s0;
    if (alike != before) __syncthreads();   // (a thread's places in shared memory change)
    before = alike;
    const int place = alike ? K / V * V : 0;   // of the elements outside pieces
    const int head = alike ? min(K, (16 - s0) % 16 / (int)sizeof(T)) : K, pieces = (K - head) / V;
    const int after = head + pieces * V, single = K - pieces * V;   // elements outside pieces
    float s[2] = {0.0f, 0.0f};
    // n neighbouring elements from column c on
    auto first = [&](auto& vx, auto& vr, int n, int c) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (i >= n) break;
        float f = to_float(vx.v[i]);
        if (kBackward) {
          s[1] = fmaf(to_float(vr.v[i]) * gamma[padded<T>(c + i)], f, s[1]);
        } else if (r) {
          from_float(vx.v[i], f + to_float(vr.v[i]));
          f = to_float(vx.v[i]);
        }
        s[0] = fmaf(f, f, s[0]);
      }
    };
#pragma unroll 2
    for (int p = tid; p < pieces; p += step) {
      const int c = head + p * V;
      Piece vx = *reinterpret_cast<const Piece*>(x + c), vr;
      if (kBackward || r) vr = *reinterpret_cast<const Piece*>(r + c);
      first(vx, vr, V, c);
      if (h) *reinterpret_cast<Piece*>(h + c) = vx;
      if (keep) {
        reinterpret_cast<Piece*>(hs)[p] = vx;
        if (kBackward) reinterpret_cast<Piece*>(ds)[p] = vr;
      }
    }
    for (int i = tid; i < single; i += step) {
      const int c = i < head ? i : after + i - head;
      Piece vx, vr;
      vx.v[0] = x[c];
      if (kBackward || r) vr.v[0] = r[c];
      first(vx, vr, 1, c);
      if (h) h[c] = vx.v[0];
      if (keep) {
        hs[place + i] = vx.v[0];
        if (kBackward) ds[place + i] = vr.v[0];
      }
    }
    lane_sums(s, 32);
    if ((tid & 31) == 0) {
      part[turn][tid >> 5] = s[0];
      part[turn][16 + (tid >> 5)] = s[1];
    }
    __syncthreads();
    s[0] = s[1] = 0.0f;
    for (int i = 0; i < warps; ++i) {
      s[0] += part[turn][i];
      s[1] += part[turn][16 + i];
    }
    const float inv = inverse(a, s[0]), m = inv * inv * (s[1] * a.inv_K);
    auto second = [&](auto& vx, const auto& vd, const auto& ve, int n, int c) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (i >= n) break;
        const float f = to_float(vx.v[i]), w = gamma[padded<T>(c + i)];
        float o = f * inv * w;
        if (kBackward) {
          const float d = to_float(vd.v[i]);
          acc[padded<T>(c + i)] = fmaf(d, f * inv, acc[padded<T>(c + i)]);
          o = inv * fmaf(-f, m, d * w);
          if (e) o += to_float(ve.v[i]);
        }
        from_float(vx.v[i], o);
      }
    };
    const T* again = h ? h : x;   // (this thread's own elements, where they are not kept)
#pragma unroll 2
    for (int p = tid; p < pieces; p += step) {
      const int c = head + p * V;
      Piece vx = keep ? reinterpret_cast<const Piece*>(hs)[p] : *reinterpret_cast<const Piece*>(again + c), vd, ve;
      if (kBackward) vd = keep ? reinterpret_cast<const Piece*>(ds)[p] : *reinterpret_cast<const Piece*>(r + c);
      if (e) ve = *reinterpret_cast<const Piece*>(e + c);
      second(vx, vd, ve, V, c);
      *reinterpret_cast<Piece*>(y + c) = vx;
    }
    for (int i = tid; i < single; i += step) {
      const int c = i < head ? i : after + i - head;
      Piece vx, vd, ve;
      vx.v[0] = keep ? hs[place + i] : again[c];
      if (kBackward) vd.v[0] = keep ? ds[place + i] : r[c];
      if (e) ve.v[0] = e[c];
      second(vx, vd, ve, 1, c);
      y[c] = vx.v[0];
    }
  }
  if (kBackward) {
    __syncthreads();
    for (int c = tid; c < K; c += step) a.parts[(int64_t)blockIdx.x * K + c] = acc[padded<T>(c)];
  }
}

// d_gamma: 32 columns a block, its 32 warps a share of the parts each, both added
// up in order: the same sums whatever ran first. Its launch overlaps the end of the
// kernel that leaves the parts.
__global__ void __launch_bounds__(1024) rms_norm_gamma_kernel(const float* parts, int n, int K,
                                                              float* __restrict__ d_gamma) {
  __shared__ float sums[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
  float s = 0.0f;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (col < K) {
#pragma unroll 4
    for (int i = warp; i < n; i += 32) s += __ldcg(parts + (int64_t)i * K + col);
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || col >= K) return;
  s = 0.0f;
#pragma unroll
  for (int i = 0; i < 32; ++i) s += sums[i][lane];
  d_gamma[col] = s;
}

// ------------------------------------------------------------------ host

bool sizes_ok(int type, int64_t rows, int64_t K, float eps) {
  return type_ok(type) && rows >= 0 && K >= 0 && K <= kMaxWidth && rows < (1ll << 31) && eps >= 0.0f;
}

// Whether all operands' rows are runs of eight elements on 16-byte boundaries.
struct Align {
  int64_t es;
  bool runs;
};
bool operand_ok(const void* p, int64_t ld, int64_t K, Align& al) {
  if (!p || ld < K || !aligned(p, al.es)) return false;
  al.runs = al.runs && aligned(p, 16) && ld * al.es % 16 == 0;
  return true;
}

template <typename Kernel>
bool allow_shared(Kernel kernel, int64_t bytes) {
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) == cudaSuccess) return true;
  cudaGetLastError();
  return false;
}

// Persistent blocks for many rows: P runs to a thread, at most kThreads threads. 0
// where the rows are few or too wide (the other forms take them), else the blocks.
template <int P, int kThreads, typename Kernel>
unsigned launch_rows(Kernel kernel, NormArgs& a, int64_t es, int operands, int sms, cudaStream_t s) {
  const int tpr = (int)ceil_div(a.K, P * kRun * 32) * 32;
  if (tpr > kThreads || a.rows < kRowsOfSM * sms) return 0;
  int groups = kThreads / tpr;
  if (tpr > 32 && groups > 15) groups = 15;   // named barriers
  if (groups * (tpr >> 5) > 32) groups = 32 / (tpr >> 5);
  int stages = kMaxStages;
  while (stages > 0 && ring_bytes(a.K, es, operands, stages) > kSharedOfBlock) --stages;
  if (stages < 2) return 0;
  // Each place belongs to one group, which has two or more: one row at hand, one on
  // its way. (So the groups' shares of d_gamma fit where the rows were, too.)
  if (groups > stages / 2) groups = stages / 2;
  stages -= stages % groups;
  const int64_t smem = ring_bytes(a.K, es, operands, stages);
  if (!allow_shared(kernel, kSharedOfBlock)) return 0;
  a.tpr = tpr, a.groups = groups, a.stages = stages;
  a.wait_limit_ns = wait_limit_ns(), a.status = device_status_word(), a.test_stall = test_stall_on() == 1;
  if (!a.status) return 0;
  kernel<<<sms, tpr * groups, smem, s>>>(a);
  return (unsigned)sms;
}

// The form for any alignment: its blocks, at most `most`; 0 if the launch failed.
template <typename T, bool kBackward>
unsigned launch_any(NormArgs& a, int64_t most, int sms, cudaStream_t s) {
  auto kernel = rms_norm_any_kernel<T, kBackward>;
  constexpr int64_t room = kSharedOfBlock - 1024;   // beside the kernel's own
  const int64_t operands = kBackward ? 2 : 1, fixed = operands * gamma_bytes<T>(a.K), kept = operands * row_bytes<T>(a.K);
  a.stages = fixed + kept <= room;
  const int64_t smem = fixed + (a.stages ? kept : 0);
  if (smem > room || !allow_shared(kernel, room)) return 0;
  const int threads = a.K >= 512 * 8 ? 512 : a.K >= 256 * 4 ? 256 : 128;
  int64_t fit = kSharedOfBlock / (smem + 2048);      // blocks of an SM
  if (fit > 1024 / threads) fit = 1024 / threads;
  const int64_t blocks = sms * (fit < 1 ? 1 : fit);
  const unsigned grid = (unsigned)(most < blocks ? most : blocks);
  kernel<<<grid, threads, smem, s>>>(a);
  return launch_status() == NVFP4MOE_OK ? grid : 0;
}

template <typename T>
int forward_of(NormArgs& a, const Align& al, int sms, cudaStream_t s) {
  const int64_t K = a.K;
  if (!al.runs) return launch_any<T, false>(a, a.rows, sms, s) ? NVFP4MOE_OK : NVFP4MOE_ERR_LAUNCH;
  if constexpr (sizeof(T) == 2) {
    if (K >= kWideRow && launch_rows<4, 896>(rms_norm_rows_kernel<T, 4, 896>, a, sizeof(T), a.r ? 2 : 1, sms, s))
      return launch_status();
  }
  const int P = K <= 8192 ? 2 : 4;
  const int64_t need = ceil_div(K, kRun * P);
  a.tpr = need <= 16 ? 16 : (int)ceil_div(need, 32) * 32;   // sixteen threads hold a block of codes
  a.groups = a.tpr >= 128 ? 1 : 128 / a.tpr;
  const unsigned grid = (unsigned)ceil_div(a.rows, a.groups);
  if (P == 2) rms_norm_kernel<T, 2><<<grid, a.tpr * a.groups, 0, s>>>(a);
  else rms_norm_kernel<T, 4><<<grid, a.tpr * a.groups, 0, s>>>(a);
  return launch_status();
}

constexpr int kBackwardBlocks = 1216;   // of the any-alignment form: eight to an SM
int64_t backward_parts(int64_t rows) { return rows < kBackwardBlocks ? rows : kBackwardBlocks; }

// The blocks that leave a part of d_gamma each; 0 if a launch failed.
template <typename T>
unsigned backward_of(NormArgs& a, const Align& al, int sms, cudaStream_t s) {
  if (al.runs && sms <= kBackwardBlocks) {
    constexpr int kP = sizeof(T) == 2 ? 4 : 2, kThreads = sizeof(T) == 2 ? 448 : 512;
    if (const unsigned n = launch_rows<kP, kThreads>(rms_norm_backward_rows_kernel<T, kP, kThreads>, a, sizeof(T),
                                                     a.dh ? 3 : 2, sms, s))
      return launch_status() == NVFP4MOE_OK ? n : 0;
  }
  return launch_any<T, true>(a, backward_parts(a.rows), sms, s);
}

int forward(NormArgs& a, int type, int64_t K, bool quantize, void* stream) {
  NVFP4_CHECK(sizes_ok(type, a.rows, K, a.eps) && (!quantize || K % 16 == 0), NVFP4MOE_ERR_UNSUPPORTED);
  if (a.rows == 0 || K == 0) return NVFP4MOE_OK;
  Align al{type_bytes(type), K % kRun == 0 && aligned(a.gamma, 16)};
  NVFP4_CHECK(a.gamma && aligned(a.gamma, 4) && operand_ok(a.x, a.ldx, K, al) &&
                  (a.r ? operand_ok(a.r, a.ldr, K, al) && operand_ok(a.h, a.ldh, K, al) : a.h == nullptr) &&
                  (!a.y || operand_ok(a.y, a.ldy, K, al)),
              NVFP4MOE_ERR_INVALID);
  NVFP4_CHECK(quantize ? al.runs && a.codes && a.sf && aligned(a.codes, 16) && aligned(a.sf, 4) : a.y != nullptr,
              NVFP4MOE_ERR_INVALID);
  const int sms = device_num_sms();
  NVFP4_CHECK(sms > 0, NVFP4MOE_ERR_LAUNCH);
  a.K = (int)K;
  a.inv_K = 1.0f / (float)K;
  cudaStream_t s = as_stream(stream);
  if (type == NVFP4MOE_BF16) return forward_of<__nv_bfloat16>(a, al, sms, s);
  if (type == NVFP4MOE_F16) return forward_of<__half>(a, al, sms, s);
  return forward_of<float>(a, al, sms, s);
}

}  // namespace
}  // namespace nvfp4moe

using namespace nvfp4moe;

extern "C" int rms_norm(const void* x, int type, int64_t rows, int64_t K, int64_t ldx, const void* residual,
                        int64_t ldr, const float* gamma, float eps, void* h, int64_t ldh, void* y, int64_t ldy,
                        void* stream) {
  NormArgs a{};
  a.x = x, a.ldx = ldx, a.r = residual, a.ldr = ldr, a.gamma = gamma, a.eps = eps, a.rows = rows;
  a.h = h, a.ldh = ldh, a.y = y, a.ldy = ldy;
  return forward(a, type, K, false, stream);
}

extern "C" int fp8_rms_norm_quantize(const void* x, int type, int64_t rows, int64_t K, int64_t ldx,
                                     const void* residual, int64_t ldr, const float* gamma, float eps, void* h,
                                     int64_t ldh, void* y, int64_t ldy, uint8_t* codes, float* sf, void* stream) {
  NormArgs a{};
  a.x = x, a.ldx = ldx, a.r = residual, a.ldr = ldr, a.gamma = gamma, a.eps = eps, a.rows = rows;
  a.h = h, a.ldh = ldh, a.y = y, a.ldy = ldy, a.codes = codes, a.sf = sf;
  return forward(a, type, K, true, stream);
}

extern "C" size_t rms_norm_backward_workspace_size(int64_t rows, int64_t K) {
  if (rows < 0 || K < 0 || K > kMaxWidth) return 0;
  if (rows == 0 || K == 0) return 0;
  return (size_t)(backward_parts(rows) * K * 4);
}

extern "C" int rms_norm_backward(const void* dy, int type, int64_t rows, int64_t K, int64_t lddy, const void* h,
                                 int64_t ldh, const float* gamma, float eps, const void* dh, int64_t lddh, void* dx,
                                 int64_t lddx, float* d_gamma, void* ws, size_t ws_bytes, void* stream) {
  NVFP4_CHECK(sizes_ok(type, rows, K, eps), NVFP4MOE_ERR_UNSUPPORTED);
  if (K == 0) return NVFP4MOE_OK;
  NVFP4_CHECK(d_gamma && aligned(d_gamma, 4), NVFP4MOE_ERR_INVALID);
  cudaStream_t s = as_stream(stream);
  if (rows == 0)
    return cudaMemsetAsync(d_gamma, 0, K * 4, s) == cudaSuccess ? NVFP4MOE_OK : NVFP4MOE_ERR_LAUNCH;
  Align al{type_bytes(type), K % kRun == 0 && aligned(gamma, 16)};
  NVFP4_CHECK(gamma && aligned(gamma, 4) && operand_ok(dy, lddy, K, al) && operand_ok(h, ldh, K, al) &&
                  (!dh || operand_ok(dh, lddh, K, al)) && operand_ok(dx, lddx, K, al),
              NVFP4MOE_ERR_INVALID);
  NVFP4_CHECK(ws && ws_bytes >= rms_norm_backward_workspace_size(rows, K) && aligned(ws, 4), NVFP4MOE_ERR_WORKSPACE);
  const int sms = device_num_sms();
  NVFP4_CHECK(sms > 0, NVFP4MOE_ERR_LAUNCH);
  NormArgs a{};
  a.dy = dy, a.lddy = lddy, a.dh = dh, a.lddh = lddh, a.h = const_cast<void*>(h), a.ldh = ldh, a.y = dx, a.ldy = lddx;
  a.gamma = gamma, a.eps = eps, a.rows = rows, a.K = (int)K, a.inv_K = 1.0f / (float)K;
  a.parts = static_cast<float*>(ws);
  const unsigned parts = type == NVFP4MOE_BF16  ? backward_of<__nv_bfloat16>(a, al, sms, s)
                         : type == NVFP4MOE_F16 ? backward_of<__half>(a, al, sms, s)
                                                : backward_of<float>(a, al, sms, s);
  NVFP4_CHECK(parts, NVFP4MOE_ERR_LAUNCH);
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)ceil_div(K, 32), 1, 1);
  cfg.blockDim = dim3(1024, 1, 1);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, rms_norm_gamma_kernel, (const float*)a.parts, (int)parts, (int)K, d_gamma);
  return launch_status();
}
