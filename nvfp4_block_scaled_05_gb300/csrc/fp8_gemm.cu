// Block-scaled 8-bit matrix product for sm_103a, dense and grouped by expert:
//   C[m, n] = sum_b sa[m, b] * sw[n / 128, b] * sum_{k in block b} A[m, k] * W[n, k]
// with E4M3 codes, one f32 activation scale per row and 128 elements of K, and
// one f32 weight scale per 128 x 128 block.
//
// The f32 scales cannot be applied by the tensor core, so each 128-element
// block of K is one partial product: four tcgen05.mma kind::f8f6f4 (M=128,
// N=256, K=32) into one of two tensor-memory buffers, which the epilogue warps
// read back, scale and add to f32 accumulators in registers while the tensor
// core fills the other buffer. The products of a block are summed by the
// tensor core, the blocks in f32 in ascending order.
//
// Tile: 128 activation rows of one group x 256 weight rows; a stage is one
// block of K, 128 bytes of every operand row (one 128-byte swizzle row).
// Warp roles (320 threads, one CTA per SM):
//   warp 0     TMA producer, a ring of 4 stages of 48 KB
//   warp 1     TMEM owner; one lane issues the MMAs
//   warps 2-9  epilogue, two warps per TMEM lane quadrant (128 columns each)
// Tiles are ordered group-major, then weight tile, then activation tile, so
// the activation tiles that share a weight tile run at the same time and it
// leaves HBM once.
//
// Every wait is bounded: a wait that exceeds the limit sets the device status
// word, raises a shared abort flag that ends the other roles' loops, and the
// CTA then waits (with a fixed bound) for its own copies and tensor-core work
// in flight, frees its tensor memory and returns.
#include "common.cuh"

#include <cuda_fp16.h>

namespace nvfp4moe {
namespace {

constexpr int BM = 128;
constexpr int BN = 256;
constexpr int BK = 128;                  // K elements (bytes) per stage: one scale block
constexpr int STAGES = 4;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (2 + kEpiWarps);
constexpr int A_BYTES = BM * BK;         // 16 KB
constexpr int B_BYTES = BN * BK;         // 32 KB
constexpr int OFF_B = STAGES * A_BYTES;
constexpr int OFF_BAR = OFF_B + STAGES * B_BYTES;
constexpr int OFF_MISC = OFF_BAR + 256;
constexpr int OFF_SCHED = OFF_MISC + 64;
constexpr uint32_t TMEM_COLS = 512;      // two accumulator buffers of 256 columns
constexpr int kMaxGroups = 1024;

struct Params {
  const float* a_sf;          // (M, KB)
  const float* w_sf;          // (E, NB, KB)
  const int32_t* offsets;     // (E + 1) rows of the groups, or null: one group of all rows
  int M, N, K, E;
  int KB, NB;                 // blocks of 128 along K and N
  void* c;
  int c_type;
  int64_t ldc;
  int c_32B;                  // c and ldc allow 32-byte stores
  uint64_t wait_limit_ns;
  int* status;
  int test_stall;             // test hook: the MMA issuer first waits on a barrier nobody arrives on
};

// First row of every group (start[E] = the end of the last) and first tile of
// every group. Bounds outside [0, M] or out of order are clamped, so that no
// tile reaches past the operands whatever the offsets hold.
struct Sched {
  const int32_t* start;       // [2E]: first row, rows
  const int32_t* tile_start;  // [E + 1]
  int E, NT, N;
  __device__ __forceinline__ void decode(int t, int& e, int& nb, int& row0, int& rows, int& ncols) const {
    int lo = 0, hi = E - 1;
    while (lo < hi) {  // largest e with tile_start[e] <= t
      const int mid = (lo + hi + 1) >> 1;
      if (tile_start[mid] <= t) lo = mid;
      else hi = mid - 1;
    }
    e = lo;
    const int mt = (tile_start[e + 1] - tile_start[e]) / NT;
    const int local = t - tile_start[e];
    nb = local / mt;
    const int mb = local - nb * mt;
    row0 = start[2 * e] + mb * BM;
    rows = min(BM, start[2 * e + 1] - mb * BM);
    ncols = min(BN, N - nb * BN);
  }
};

// Instruction descriptor: kind::f8f6f4, A and B E4M3 K-major, f32 accumulate.
__device__ constexpr uint32_t idesc_e4m3(int M, int N) {
  return (1u << 4)                                  // D format: f32
         | (static_cast<uint32_t>(N >> 3) << 17)    // N / 8
         | (static_cast<uint32_t>(M >> 4) << 24);   // M / 16
}

__device__ __forceinline__ void tc_mma_f8(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 32 consecutive columns of this thread's TMEM lane, waited for.
__device__ __forceinline__ void tc_ld32_wait(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ uint32_t pack2(const __nv_bfloat16*, float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack2(const __half*, float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put(__half* p, float v) { *p = __float2half_rn(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }

// The first n of 16 values to out: 32-byte stores where the row allows them.
template <typename T>
__device__ __forceinline__ void store16(T* out, const float* v, int n, bool wide) {
  if (wide && n >= 16) {
    if constexpr (sizeof(T) == 2) {
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = pack2(out, v[2 * i], v[2 * i + 1]);
      st_global_32B_stream(out, w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        st_global_32B_stream(out + 8 * h, __float_as_uint(v[8 * h]), __float_as_uint(v[8 * h + 1]),
                             __float_as_uint(v[8 * h + 2]), __float_as_uint(v[8 * h + 3]),
                             __float_as_uint(v[8 * h + 4]), __float_as_uint(v[8 * h + 5]),
                             __float_as_uint(v[8 * h + 6]), __float_as_uint(v[8 * h + 7]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < n) put(out + i, v[i]);
  }
}

template <typename T>
__device__ __forceinline__ void store_row(T* out, const float (&acc)[128], int n, bool wide) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (16 * j < n) store16(out + 16 * j, acc + 16 * j, n - 16 * j, wide);
}

__global__ void __launch_bounds__(kThreads, 1)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap tm_a16, const __grid_constant__ CUtensorMap tm_a32,
                    const __grid_constant__ CUtensorMap tm_a64, const __grid_constant__ CUtensorMap tm_a128,
                    const __grid_constant__ CUtensorMap tm_b128, const __grid_constant__ CUtensorMap tm_b256,
                    const Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sbase = smem_addr(smem);
  const uint32_t bar_full = sbase + OFF_BAR;            // STAGES: a stage's tiles landed
  const uint32_t bar_empty = bar_full + STAGES * 8;     // STAGES: its MMAs are done
  const uint32_t bar_accf = bar_empty + STAGES * 8;     // 2: a buffer holds a block's products
  const uint32_t bar_acce = bar_accf + 16;              // 2: the epilogue has read it
  const uint32_t bar_aux = bar_acce + 16;               // MMA drain on abort
  const uint32_t bar_never = bar_aux + 8;               // never arrived on (failure-path test)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_MISC + 4);
  int32_t* start = reinterpret_cast<int32_t*>(smem + OFF_SCHED);
  int32_t* tile_start = start + 2 * p.E;
  const int E = p.E, NT = (p.N + BN - 1) / BN;

  // --- schedule: rows of every group, then the prefix sum of its tiles
  for (int e = tid; e < E; e += kThreads) {
    int lo = 0, hi = p.M;
    if (p.offsets) {
      lo = min(max(p.offsets[e], 0), p.M);
      hi = min(max(p.offsets[e + 1], lo), p.M);
    }
    start[2 * e] = lo;
    start[2 * e + 1] = hi - lo;
  }
  if (tid == 32) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(bar_full + 8 * s, 1);
      mbar_init(bar_empty + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar_accf + 8 * b, 1);
      mbar_init(bar_acce + 8 * b, kEpiWarps);
    }
    mbar_init(bar_aux, 1);
    mbar_init(bar_never, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(tmem_slot), TMEM_COLS);
    tmem_relinquish();
  }
  __syncthreads();
  if (warp == 0) {
    int carry = 0;
    for (int base = 0; base < E; base += 32) {
      const int e = base + lane;
      const int mt = e < E ? (start[2 * e + 1] + BM - 1) / BM : 0;
      int incl = mt;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, incl, d);
        if (lane >= d) incl += y;
      }
      if (e < E) tile_start[e] = (carry + incl - mt) * NT;
      carry += __shfl_sync(0xFFFFFFFFu, incl, 31);
    }
    if (lane == 0) tile_start[E] = carry * NT;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int total = tile_start[E];
  const Sched sch{start, tile_start, E, NT, p.N};
  const int KB = p.KB;

  if (warp == 0 && lane == 0) {
    // ---------------------------------------------------------------- producer
    // A weight tile read by one activation tile only is streamed (evict
    // first); one that several read keeps normal priority.
    const uint64_t pol_w1 = l2_policy_evict_first();
    const uint64_t pol_wn = l2_policy_evict_normal();
    const uint64_t pol_a = l2_policy_evict_last();
    uint32_t stage = 0, phase = 0, filled = 0, fill_phase = 0;
    bool ok = true;
    for (int t = blockIdx.x; ok && t < total; t += gridDim.x) {
      int e, nb, row0, rows, ncols;
      sch.decode(t, e, nb, row0, rows, ncols);
      const CUtensorMap* tma = rows <= 16 ? &tm_a16 : rows <= 32 ? &tm_a32 : rows <= 64 ? &tm_a64 : &tm_a128;
      const int box = rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
      // rows of the box past the group or the weight's last row are multiplied
      // too; their products stay in rows and columns that are not stored
      const CUtensorMap* tmb = ncols <= 128 ? &tm_b128 : &tm_b256;
      const uint32_t tx = (uint32_t)(box * BK + (ncols <= 128 ? 128 : 256) * BK);
      const int b_row = e * p.N + nb * BN;
      const uint64_t pol_w = tile_start[e + 1] - tile_start[e] > NT ? pol_wn : pol_w1;
      for (int kb = 0; kb < KB; ++kb) {
        if (!wait_bounded(bar_empty + 8 * stage, phase ^ 1, abort_flag, p.wait_limit_ns, p.status, 31)) {
          ok = false;
          break;
        }
        const uint32_t full = bar_full + 8 * stage;
        mbar_arrive_expect_tx(full, tx);
        tma_load_2d(sbase + stage * A_BYTES, tma, full, kb * BK, row0, pol_a);
        tma_load_2d(sbase + OFF_B + stage * B_BYTES, tmb, full, kb * BK, b_row, pol_w);
        filled |= 1u << stage;
        fill_phase = (fill_phase & ~(1u << stage)) | (phase << stage);
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    if (!ok)   // copies still in flight complete before the CTA may exit
      for (int s = 0; s < STAGES; ++s)
        if ((filled >> s) & 1u) drain_wait(bar_full + 8 * s, (fill_phase >> s) & 1u);
  } else if (warp == 1 && lane == 0) {
    // ---------------------------------------------------------------- MMA issuer
    uint32_t stage = 0, phase = 0, g = 0;
    bool ok = true, issued = false;
    const uint64_t adesc0 = sdesc_kmajor_sw128(sbase);
    const uint64_t bdesc0 = sdesc_kmajor_sw128(sbase + OFF_B);
    if (p.test_stall && (int)blockIdx.x < total)
      ok = wait_bounded(bar_never, 0, abort_flag, p.wait_limit_ns, p.status, 32);
    for (int t = blockIdx.x; ok && t < total; t += gridDim.x) {
      int e, nb, row0, rows, ncols;
      sch.decode(t, e, nb, row0, rows, ncols);
      const uint32_t idesc = idesc_e4m3(BM, (ncols + 15) / 16 * 16);
      for (int kb = 0; kb < KB; ++kb, ++g) {
        const uint32_t buf = g & 1u;
        if (!wait_bounded(bar_acce + 8 * buf, ((g >> 1) & 1u) ^ 1u, abort_flag, p.wait_limit_ns, p.status, 33) ||
            !wait_bounded(bar_full + 8 * stage, phase, abort_flag, p.wait_limit_ns, p.status, 34)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t ad = adesc0 + ((stage * A_BYTES) >> 4);
        const uint64_t bd = bdesc0 + ((stage * B_BYTES) >> 4);
#pragma unroll
        for (int kk = 0; kk < BK / 32; ++kk)   // 32 bytes of every row further per step
          tc_mma_f8(tmem + buf * BN, ad + 2 * kk, bd + 2 * kk, idesc, kk != 0 ? 1u : 0u);
        issued = true;
        tc_commit(bar_empty + 8 * stage);
        tc_commit(bar_accf + 8 * buf);
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    if (!ok && issued) {   // tensor-core work in flight completes before the tensor memory is freed
      tc_commit(bar_aux);
      drain_wait(bar_aux, 0);
    }
  } else if (warp >= 2) {
    // ---------------------------------------------------------------- epilogue
    const int quad = warp & 3;              // TMEM lane quadrant this warp may access
    const int half = (warp - 2) >> 2;       // columns [128 * half, 128 * half + 128): one weight scale a block
    const int row = quad * 32 + lane;
    const uint32_t taddr = tmem + (static_cast<uint32_t>(quad * 32) << 16) + half * 128;
    uint32_t g = 0;
    bool ok = true;
    for (int t = blockIdx.x; ok && t < total; t += gridDim.x) {
      int e, nb, row0, rows, ncols;
      sch.decode(t, e, nb, row0, rows, ncols);
      const bool live = quad * 32 < rows && half * 128 < ncols;   // the whole warp
      const bool active = row < rows && half * 128 < ncols;
      const int64_t m = row0 + min(row, rows - 1);
      const float* sa = p.a_sf + m * KB;
      const float* sw = p.w_sf + ((int64_t)e * p.NB + min(nb * 2 + half, p.NB - 1)) * KB;
      float acc[128];
#pragma unroll
      for (int i = 0; i < 128; ++i) acc[i] = 0.0f;
      float s = live ? sa[0] * sw[0] : 0.0f;
      for (int kb = 0; kb < KB; ++kb, ++g) {
        const float s_next = live && kb + 1 < KB ? sa[kb + 1] * sw[kb + 1] : 0.0f;
        const uint32_t buf = g & 1u;
        ok = wait_bounded(bar_accf + 8 * buf, (g >> 1) & 1u, abort_flag, p.wait_limit_ns, p.status, 35);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        tc_fence_after();
        if (live) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t v[32];
            tc_ld32_wait(taddr + buf * BN + 32 * c, v);
#pragma unroll
            for (int i = 0; i < 32; ++i) acc[32 * c + i] = fmaf(__uint_as_float(v[i]), s, acc[32 * c + i]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_acce + 8 * buf);
        s = s_next;
      }
      if (!ok || !active) continue;
      const int64_t at = m * p.ldc + nb * BN + half * 128;
      const int n = min(128, ncols - half * 128);
      if (p.c_type == NVFP4MOE_BF16) store_row(static_cast<__nv_bfloat16*>(p.c) + at, acc, n, p.c_32B);
      else if (p.c_type == NVFP4MOE_F16) store_row(static_cast<__half*>(p.c) + at, acc, n, p.c_32B);
      else store_row(static_cast<float*>(p.c) + at, acc, n, p.c_32B);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

int launch(const uint8_t* a_codes, int64_t lda, const uint8_t* w_codes, int64_t ldw, Params& p, void* stream) {
  CUtensorMap ma[4], mb[2];
  const int boxes[4] = {16, 32, 64, 128};
  for (int i = 0; i < 4; ++i)
    if (!make_codes_map(&ma[i], a_codes, p.M, p.K, lda, boxes[i])) return NVFP4MOE_ERR_INVALID;
  for (int i = 0; i < 2; ++i)
    if (!make_codes_map(&mb[i], w_codes, (int64_t)p.E * p.N, p.K, ldw, 128 << i)) return NVFP4MOE_ERR_INVALID;
  p.status = device_status_word();
  NVFP4_CHECK(p.status, NVFP4MOE_ERR_LAUNCH);
  p.wait_limit_ns = wait_limit_ns();
  p.test_stall = test_stall_on();
  const size_t smem = (size_t)OFF_SCHED + 4 * (3 * (size_t)p.E + 1) + 1024;
  if (cudaFuncSetAttribute(fp8_gemm_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return launch_status();
  const int64_t most = (ceil_div(p.M, BM) + (p.E < p.M ? p.E : p.M)) * ceil_div(p.N, BN);   // upper bound of the tiles
  const int sms = device_num_sms();
  NVFP4_CHECK(sms > 0, NVFP4MOE_ERR_LAUNCH);
  const unsigned grid = (unsigned)(most < sms ? most : sms);
  fp8_gemm_kernel<<<grid, kThreads, smem, as_stream(stream)>>>(ma[0], ma[1], ma[2], ma[3], mb[0], mb[1], p);
  return launch_status();
}

int gemm(const uint8_t* a_codes, const float* a_sf, int64_t M, int64_t lda, const uint8_t* w_codes, const float* w_sf,
         const int32_t* offsets, int E, int64_t N, int64_t K, int64_t ldw, void* c, int c_type, int64_t ldc,
         void* stream) {
  NVFP4_CHECK(E >= 1 && E <= kMaxGroups && M >= 0 && N >= 0 && K >= 1 && M < (1ll << 31) - BM && K < (1ll << 31) - BK &&
                  E * N < (1ll << 31) - BN,
              NVFP4MOE_ERR_UNSUPPORTED);
  NVFP4_CHECK(c_type == NVFP4MOE_BF16 || c_type == NVFP4MOE_F16 || c_type == NVFP4MOE_F32, NVFP4MOE_ERR_UNSUPPORTED);
  if (M == 0 || N == 0) return NVFP4MOE_OK;
  NVFP4_CHECK((ceil_div(M, BM) + E) * ceil_div(N, BN) < (1ll << 31), NVFP4MOE_ERR_UNSUPPORTED);
  NVFP4_CHECK(a_codes && a_sf && w_codes && w_sf && c, NVFP4MOE_ERR_INVALID);
  NVFP4_CHECK(lda >= K && ldw >= K && lda % 16 == 0 && ldw % 16 == 0 && ldc >= N, NVFP4MOE_ERR_INVALID);
  const int es = c_type == NVFP4MOE_F32 ? 4 : 2;
  NVFP4_CHECK(aligned(a_codes, 16) && aligned(w_codes, 16) && aligned(a_sf, 4) && aligned(w_sf, 4) && aligned(c, es),
              NVFP4MOE_ERR_INVALID);
  Params p{};
  p.a_sf = a_sf;
  p.w_sf = w_sf;
  p.offsets = offsets;
  p.M = (int)M;
  p.N = (int)N;
  p.K = (int)K;
  p.E = E;
  p.KB = (int)ceil_div(K, BK);
  p.NB = (int)ceil_div(N, 128);
  p.c = c;
  p.c_type = c_type;
  p.ldc = ldc;
  p.c_32B = aligned(c, 32) && ldc * es % 32 == 0;
  return launch(a_codes, lda, w_codes, ldw, p, stream);
}

}  // namespace
}  // namespace nvfp4moe

using namespace nvfp4moe;

extern "C" int fp8_linear(const uint8_t* a_codes, const float* a_sf, int64_t M, int64_t lda, const uint8_t* w_codes,
                          const float* w_sf, int64_t N, int64_t K, int64_t ldw, void* c, int c_type, int64_t ldc,
                          void* stream) {
  return gemm(a_codes, a_sf, M, lda, w_codes, w_sf, nullptr, 1, N, K, ldw, c, c_type, ldc, stream);
}

extern "C" int fp8_grouped_gemm(const uint8_t* a_codes, const float* a_sf, int64_t M, int64_t lda,
                                const uint8_t* w_codes, const float* w_sf, const int32_t* offsets, int E, int64_t N,
                                int64_t K, int64_t ldw, void* c, int c_type, int64_t ldc, void* stream) {
  NVFP4_CHECK(offsets || M == 0, NVFP4MOE_ERR_INVALID);
  return gemm(a_codes, a_sf, M, lda, w_codes, w_sf, offsets, E, N, K, ldw, c, c_type, ldc, stream);
}
