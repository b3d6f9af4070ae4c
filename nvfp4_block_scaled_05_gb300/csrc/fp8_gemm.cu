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
// Warp roles (384 threads, one CTA per SM):
//   warp 0      TMA producer, a ring of 4 stages of 48 KB
//   warp 1      TMEM owner; issues the MMAs
//   warps 2-3   the factors sa * sw of every row and block, into a ring in
//               shared memory
//   warps 4-11  epilogue, two warps per TMEM lane quadrant (128 columns each)
// Tiles are ordered group-major, then weight tile, then activation tile, so
// the activation tiles that share a weight tile run at the same time and it
// leaves HBM once.
//
// Every wait is bounded: a wait that exceeds the limit sets the device status
// word and raises a shared abort flag that ends the other roles' loops. Once
// all roles have ended, the CTA waits (with a fixed bound) for its own copies
// and tensor-core work in flight, whichever role gave up, frees its tensor
// memory and returns. A tile whose sums are not complete is not stored, nor is
// any of it by the other CTAs of its cluster. (The flags' way to the joining
// CTAs and the checks at the end take 0.2 us of a call: 1 x 4096 x 7168 7.7 us,
// without them 7.5.)
#include "common.cuh"

#include <cuda_fp16.h>

#include <atomic>

namespace nvfp4moe {
namespace {

constexpr int BM = 128;
constexpr int BN = 256;
constexpr int BK = 128;                  // K elements (bytes) per stage: one scale block
constexpr int HN = BN / 2;               // columns of one epilogue warpgroup
constexpr int kEpiWarp0 = 4;             // the first of two epilogue warpgroups
constexpr int kThreads = 32 * (kEpiWarp0 + 8);
constexpr int STAGES = 4;
constexpr int A_BYTES = BM * BK;         // 16 KB
constexpr int B_BYTES = BN * BK;         // 32 KB
constexpr int kScaleSlots = 8;           // blocks of K whose factors are in shared memory (see bar_done)
constexpr int OFF_B = STAGES * A_BYTES;
constexpr int OFF_BAR = OFF_B + STAGES * B_BYTES;
constexpr int OFF_SCALE = OFF_BAR + 256;                       // [slot][half][row]
constexpr int OFF_MISC = OFF_SCALE + kScaleSlots * 2 * BM * 4;
constexpr int OFF_SCHED = OFF_MISC + 64;
constexpr uint32_t TMEM_COLS = 512;      // two buffers of 256 columns
constexpr int kPartBytes = BN * 4 + 16;  // a row of partial sums in shared memory; 16 bytes against bank conflicts
constexpr int kMaxSplit = 8;
constexpr int kMaxGroups = 1024;
static_assert(BM * kPartBytes <= OFF_BAR, "the partial sums lie in the ring");
constexpr int kMaxShared = 232448;       // of a CTA
constexpr int kSharedOfSM = 228 * 1024;  // each CTA on it takes 1 KB more than it asks for

// Dynamic shared memory of a kernel whose schedule of E groups starts at
// `sched`; the first 1024-byte boundary in it is offset 0.
constexpr size_t shared_bytes(int sched, int E) { return (size_t)sched + 4 * (2 * (size_t)E + 2) + 1024; }
static_assert(shared_bytes(OFF_SCHED, kMaxGroups) <= kMaxShared, "shared memory budget");

struct Params {
  const float* a_sf;          // (M, KB)
  const float* w_sf;          // (E, NB, KB)
  const int32_t* offsets;     // (E + 1) rows of the groups, or null: one group of all rows
  int M, N, K, E;
  int KB, NB;                 // blocks of 128 along K and N
  void* c;
  int c_type;
  int64_t ldc;
  int w_once;                 // few rows: every weight row is read by one tile only
  int split;                  // CTAs (a cluster) that share a tile's blocks of K
  int c_32B;                  // c and ldc allow 32-byte stores
  int c_unit;                 // bytes (2 to 16) that every row of c can be stored in units of
  uint64_t wait_limit_ns;
  int* status;
  int test_stall;             // test hook: 1: the MMA issuer first waits on a barrier nobody arrives on; 2: no factors
};

// Tiles of tm activation rows of one group x tn weight rows, ordered
// group-major, then weight tile, then activation tile.
struct Sched {
  const int32_t* bounds;      // [E + 1]: first row of every group
  const int32_t* tile_start;  // [E + 1]: first tile of every group
  int E, NT, N, tm, tn;
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
    row0 = bounds[e] + mb * tm;
    rows = min(tm, bounds[e + 1] - row0);
    ncols = min(tn, N - nb * tn);
  }
};

// The groups' bounds, by all threads, clamped to [0, M] but not yet in order.
__device__ __forceinline__ void load_bounds(const Params& p, int32_t* bounds) {
  for (int e = threadIdx.x; e <= p.E; e += blockDim.x)
    bounds[e] = p.offsets ? min(max(p.offsets[e], 0), p.M) : e == 0 ? 0 : p.M;
}

// Bounds that do not ascend become the largest so far, by one warp: whatever
// the offsets hold, the groups have no row in common, there are no more tiles
// than the host reckons with, and no tile reaches past the operands.
__device__ __forceinline__ void put_in_order(int E, int32_t* bounds) {
  if ((threadIdx.x & 31) == 0)
    for (int e = 0; e < E; ++e) bounds[e + 1] = max(bounds[e], bounds[e + 1]);
  __syncwarp();
}

// The bounds in order and the prefix sum of the groups' tiles, by one warp, 32
// groups at a time.
__device__ __forceinline__ void scan_tiles(const Sched& sch, int32_t* bounds, int32_t* tile_start) {
  const int lane = threadIdx.x & 31;
  int carry = 0;
  for (int base = 0; base < sch.E; base += 32) {
    const int e = base + lane;
    int rows = e < sch.E ? bounds[e + 1] - bounds[e] : 0;
    if (__builtin_expect(__any_sync(0xFFFFFFFFu, rows < 0), 0)) {   // (the groups before ascend, and stay as they are)
      put_in_order(sch.E, bounds);
      rows = e < sch.E ? bounds[e + 1] - bounds[e] : 0;
    }
    const int mt = (rows + sch.tm - 1) / sch.tm;
    int incl = mt;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, incl, d);
      if (lane >= d) incl += y;
    }
    if (e < sch.E) tile_start[e] = (carry + incl - mt) * sch.NT;
    carry += __shfl_sync(0xFFFFFFFFu, incl, 31);
  }
  if (lane == 0) tile_start[sch.E] = carry * sch.NT;
}

// The same, a run of neighbouring groups a lane: fewer steps (8 rows of 256
// groups, 7168 x 2048: 26.3 us against 27.8), but in the kernel with 128-row
// tiles the compiler makes a slower epilogue beside it (4096 x 4096 x 7168 103.7
// us against 102.5).
__device__ __forceinline__ void scan_tiles_by_runs(const Sched& sch, int32_t* bounds, int32_t* tile_start) {
  const int lane = threadIdx.x & 31, run = (sch.E + 31) / 32;
  const int e0 = min(lane * run, sch.E), e1 = min(e0 + run, sch.E);
  bool ascending = true;
  int tiles = 0;
  auto count = [&]() {
    tiles = 0;
    for (int e = e0; e < e1; ++e) {
      const int rows = bounds[e + 1] - bounds[e];
      ascending = ascending && rows >= 0;
      tile_start[e] = tiles;
      tiles += (rows + sch.tm - 1) / sch.tm;
    }
  };
  count();
  if (__builtin_expect(!__all_sync(0xFFFFFFFFu, ascending), 0)) {
    put_in_order(sch.E, bounds);
    count();
  }
  int incl = tiles;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, incl, d);
    if (lane >= d) incl += y;
  }
  for (int e = e0; e < e1; ++e) tile_start[e] = (incl - tiles + tile_start[e]) * sch.NT;
  if (lane == 31) tile_start[sch.E] = incl * sch.NT;
}

// Instruction descriptor: kind::f8f6f4, A and B E4M3 K-major, f32 accumulate.
__device__ constexpr uint32_t idesc_e4m3(int M, int N) {
  return (1u << 4)                                  // D format: f32
         | (static_cast<uint32_t>(N >> 3) << 17)    // N / 8
         | (static_cast<uint32_t>(M >> 4) << 24);   // M / 16
}

// True in one lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ void tc_mma_f8(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 16 consecutive columns of this thread's TMEM lane, waited for.
__device__ __forceinline__ void tc_ld16_wait(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// A converged warp's wait on a barrier, as wait_bounded, with one vote to an
// attempt; the result is the same in all lanes.
__device__ __forceinline__ bool try_wait_warp(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "vote.sync.all.pred p, p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int* abort_flag, uint64_t limit_ns,
                                          int* status, int site) {
  if (__builtin_expect(try_wait_warp(bar, parity), 1)) return true;
  uint64_t t0 = 0;
  for (uint32_t it = 1;; ++it) {
    if (try_wait_warp(bar, parity)) return true;
    if ((it & 15u) == 0) {
      bool give_up = *abort_flag != 0;
      const uint64_t now = global_timer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > limit_ns) {
        give_up = true;
        *abort_flag = 1;
        if (atomicCAS(&status[0], 0, NVFP4MOE_ERR_DEVICE_TIMEOUT) == 0) status[1] = site;
      }
      if (__any_sync(0xFFFFFFFFu, give_up)) return false;
    }
  }
}

// What a CTA has in flight when its roles have ended, left by them in shared
// memory for drain(): an abort may come from a role that waits on others'
// work, while the producer and the MMA issuer have issued all of theirs and
// ended as usual.
struct InFlight {
  uint32_t filled, fill_phase;   // stages with a copy, and the phase of its last one
  uint32_t issued;               // MMAs were issued
};

// Waits for the copies (barriers bar_full, one a stage) and MMAs of an aborted
// CTA. Called by warps 0 (whose lane 0 is the producer) and 1 (the MMA issuer,
// converged) after a barrier of the CTA that follows all roles. The CTA's shared
// memory lasts until warp 0 is through, its tensor memory until warp 1 is,
// which frees it.
__device__ __forceinline__ void drain(const InFlight& f, int warp, int lane, int stages, uint32_t bar_full,
                                      uint32_t bar_aux) {
  if (warp == 0 && lane == 0) {
    for (int s = 0; s < stages; ++s)
      if ((f.filled >> s) & 1u) drain_wait(bar_full + 8 * s, (f.fill_phase >> s) & 1u);
  } else if (warp == 1 && f.issued) {
    if (elect_one()) {   // the lane that issued them
      tc_commit(bar_aux);
      drain_wait(bar_aux, 0);
    }
    __syncwarp();
  }
}

// A word of the shared memory of a CTA of the cluster (shared::cluster address).
__device__ __forceinline__ uint32_t ld_shared_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// Four f32 from and into the shared memory of a CTA of the cluster
// (shared::cluster address).
__device__ __forceinline__ void ld_shared_cluster_v4(uint32_t addr, float* v) {
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ float ld_shared_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_shared_cluster_v4(uint32_t addr, const float* v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v[0]), "f"(v[1]), "f"(v[2]),
               "f"(v[3])
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

// Chunk j (a sector) of a row in registers, as it is stored.
template <typename T>
__device__ __forceinline__ void pack_sector(const T* type, const float (&acc)[HN], int j, uint32_t (&w)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (sizeof(T) == 2) w[i] = pack2(type, acc[16 * j + 2 * i], acc[16 * j + 2 * i + 1]);
    else w[i] = __float_as_uint(acc[8 * j + i]);
  }
}

// Lane r's row r of a warp's 32 rows, of which `rows` exist, to c + r ldc, which
// is 32-byte aligned; n columns. All lanes call it. Lanes swap sectors in pairs,
// so that a store writes 64 bytes of 16 rows and not 32 of 32, and nothing stays
// in L1 (the tile's stores take as long as three blocks of K, in which nothing is
// added up). 65536 x 7168 x 2048 in 32 groups, BF16: 820 us; without the swap 841,
// streaming stores that L1 keeps 874, without the stores 711. In fours, 128 bytes
// of 8 rows: at best another 10 us, and twice the shuffles.
template <typename T>
__device__ __forceinline__ void store_rows(T* c, int64_t ldc, const float (&acc)[HN], int rows, int n, int lane) {
  constexpr int PER = 32 / (int)sizeof(T);
  const bool odd = lane & 1;
  if (n == HN) {
    T* even_row = c + (lane & ~1) * ldc + (odd ? PER : 0);
    T* odd_row = even_row + ldc;
    const bool even_in = (lane & ~1) < rows, odd_in = (lane | 1) < rows;
#pragma unroll
    for (int j = 0; j < HN / PER; j += 2) {
      uint32_t a[8], b[8];
      pack_sector(c, acc, j, a);
      pack_sector(c, acc, j + 1, b);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, odd ? a[i] : b[i], 1);
        a[i] = odd ? got : a[i];
        b[i] = odd ? b[i] : got;
      }
      if (even_in) st_global_32B_no_l1(even_row + PER * j, a);
      if (odd_in) st_global_32B_no_l1(odd_row + PER * j, b);
    }
  } else if (lane < rows) {
#pragma unroll
    for (int j = 0; j < HN / PER; ++j) {
      T* out = c + lane * ldc + PER * j;
      if (PER * (j + 1) <= n) {
        uint32_t w[8];
        pack_sector(c, acc, j, w);
        st_global_32B_no_l1(out, w);
      } else {
#pragma unroll
        for (int i = 0; i < PER; ++i)
          if (PER * j + i < n) put(out + i, acc[PER * j + i]);
      }
    }
  }
}

// Eight values of a row of C from column `col` of `ncols` on, in the units that
// the rows allow (ncols is whole units).
template <typename U, typename T>
__device__ __forceinline__ void store_units(T* out, const T (&v)[8], int n) {
  constexpr int PER = sizeof(U) / sizeof(T) > 0 ? sizeof(U) / sizeof(T) : 1;
#pragma unroll
  for (int i = 0; i < 8; i += PER)
    if (i < n) *reinterpret_cast<U*>(out + i) = *reinterpret_cast<const U*>(v + i);
}

template <typename T>
__device__ __forceinline__ void store8(T* out, const float (&f)[8], int n, int unit) {
  alignas(16) T v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) put(v + i, f[i]);
  if (unit == 16) store_units<uint4>(out, v, n);
  else if (unit == 8) store_units<uint2>(out, v, n);
  else if (unit == 4 || sizeof(T) == 4) store_units<uint32_t>(out, v, n);
  else store_units<uint16_t>(out, v, n);
}

// w[i] = w[i + N] where `on`, for a lane each.
template <int N, int W>
__device__ __forceinline__ void shift_words(uint32_t (&w)[W], bool on) {
#pragma unroll
  for (int i = 0; i + N < W; ++i) w[i] = on ? w[i + N] : w[i];
}

// The first n values of a row to out, which is aligned to an element only. A
// store for each would touch 32 rows at a time (4096 x 4095 x 2048, BF16, took
// 183 us; rows passed on in 32-byte pieces through shared memory 54; this 39.3;
// 4096 columns and store_rows 37), so the row leaves in whole sectors: 2, 4, 8
// and 16 bytes as they are needed to reach a 32-byte boundary, then whole
// sectors of the values moved down by as many registers, and the rest in 16, 8,
// 4 and 2 bytes. (Where fewer bytes are left than a step stores, the steps end
// and they are the rest.)
template <typename T>
__device__ __forceinline__ void store_row_shifted(T* out, const float (&acc)[HN], int n) {
  constexpr int W = HN * (int)sizeof(T) / 4;
  uint32_t w[W];
  uint8_t* c = reinterpret_cast<uint8_t*>(out);
  int left = n * (int)sizeof(T);
#pragma unroll
  for (int i = 0; i < W; ++i) {
    if constexpr (sizeof(T) == 2) w[i] = pack2(out, acc[2 * i], acc[2 * i + 1]);
    else w[i] = __float_as_uint(acc[i]);
  }
  auto step = [&](int bytes) {
    const bool on = (reinterpret_cast<uintptr_t>(c) & bytes) && left >= bytes;
    c += on ? bytes : 0;
    left -= on ? bytes : 0;
    return on;
  };
  if constexpr (sizeof(T) == 2) {
    const bool on = step(2);
    if (on) *reinterpret_cast<uint16_t*>(c - 2) = (uint16_t)w[0];
    const uint32_t sel = on ? 0x5432 : 0x3210;
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = __byte_perm(w[i], w[i + 1 < W ? i + 1 : i], sel);
  }
  uint32_t t[8];   // the first, then the last words, less than a sector
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = w[i];
  const bool on1 = step(4);
  if (on1) *reinterpret_cast<uint32_t*>(c - 4) = t[0];
  shift_words<1>(t, on1);
  const bool on2 = step(8);
  if (on2) *reinterpret_cast<uint2*>(c - 8) = make_uint2(t[0], t[1]);
  shift_words<2>(t, on2);
  const bool on4 = step(16);
  if (on4) *reinterpret_cast<uint4*>(c - 16) = make_uint4(t[0], t[1], t[2], t[3]);
#pragma unroll
  for (int j = 0; j < W / 8; ++j) {
    uint32_t v[15];   // moved eight at a time: all at once would need registers for them twice
#pragma unroll
    for (int i = 0; i < 15; ++i) v[i] = 8 * j + i < W ? w[8 * j + i] : 0;
    shift_words<4>(v, on4);
    shift_words<2>(v, on2);
    shift_words<1>(v, on1);
    if (left >= 32 * (j + 1)) st_global_32B_no_l1(c + 32 * j, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = left >= 32 * j ? v[i] : t[i];
  }
  c += left & ~31;
  if (left & 16) *reinterpret_cast<uint4*>(c) = make_uint4(t[0], t[1], t[2], t[3]);
  shift_words<4>(t, left & 16);
  c += left & 16;
  if (left & 8) *reinterpret_cast<uint2*>(c) = make_uint2(t[0], t[1]);
  shift_words<2>(t, left & 8);
  c += left & 8;
  if (left & 4) *reinterpret_cast<uint32_t*>(c) = t[0];
  shift_words<1>(t, left & 4);
  if constexpr (sizeof(T) == 2) {
    c += left & 4;
    if (left & 2) *reinterpret_cast<uint16_t*>(c) = (uint16_t)t[0];
  }
}

// The parts of a tile's sums, one from each of the `split` CTAs of a cluster
// that share its blocks of K. Row r of the tile is joined by CTA r / per, which
// adds the parts in the order of the blocks. Where a thread holds a row (the
// 128-row tiles), every CTA stores its part of it straight into the owner's
// shared memory, at slot `rank` (kPull false); where a thread holds a column
// (few rows), whose stores would be four bytes each, the parts stay with the
// CTAs that made them and the owner reads them there (kPull). Measured, 128 x
// 512 x 2048 as two 128-row tiles in 2, 4 and 8 parts: 12.7, 12.6 and 12.8 us,
// read by the owner 12.8, 13.6 and 16.6; few rows, 333 x 1111 x 2000 in 2
// parts: 9.5 us, stored by the makers 11.9.
struct Parts {
  uint32_t base;   // shared memory of this CTA
  int pitch;       // bytes of a staged row
  int per;         // rows that one CTA joins
  int rank, split;
  uint32_t abort_flag;   // shared memory of this CTA
  // where this CTA's part of a row goes that is joined by its owner
  __device__ __forceinline__ uint32_t slot(int row) const {
    return mapa_shared(base + (rank * per + row % per) * pitch, row / per);
  }
};

// C's rows [row0, row0 + rows), columns [col0, col0 + ncols) of those that this
// CTA joins: eight columns of a row by one thread, the parts all on their way
// at once (a remote load takes about a microsecond). Pulled, the eight are
// neighbours, for few remote loads. Where the parts are here they are TN / 8
// apart, so that a warp's stores are neighbours at any alignment (500 x 1023 x
// 7168, f32: 17.2 us against 20.2; x 1024 17.2 against 17.8; few rows, one part,
// 64 x 8191 x 512 6.5 against 9.5, 600 x 512 x 496 6.3 against 7.0).
template <typename T, int TN, bool kPull>
__device__ __forceinline__ void join_parts(const Params& p, const Parts& parts, int row0, int rows, int col0, int ncols,
                                           int threads) {
  constexpr int STEP = kPull ? 1 : TN / 8;
  const int first = parts.rank * parts.per, mine = min(parts.per, rows - first);
  // pulled: lane r learns whether CTA r gave up, in which case nothing is stored
  uint32_t aborted = 0;
  if constexpr (kPull) {
    const int lane = threadIdx.x & 31;
    if (lane < parts.split) aborted = ld_shared_cluster_u32(mapa_shared(parts.abort_flag, lane));
  }
  for (int base = 0; base < mine * (TN / 8); base += threads) {
    const int i = base + threadIdx.x;
    const int row = i / (TN / 8), col = i % (TN / 8) * (kPull ? 8 : 1);
    const bool in = row < mine && col < ncols;
    if (!kPull && !in) continue;
    float w[kMaxSplit][8], v[8];
#pragma unroll
    for (int r = 0; r < kMaxSplit; ++r) {
      if (r < parts.split && in) {
        const uint32_t at = parts.base + (kPull ? first + row : r * parts.per + row) * parts.pitch + col * 4;
        if constexpr (kPull) {
          const uint32_t from = parts.split > 1 ? mapa_shared(at, r) : at;
          ld_shared_cluster_v4(from, w[r]);
          ld_shared_cluster_v4(from + 16, w[r] + 4);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) w[r][k] = ld_shared_f32(at + 4 * STEP * k);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      v[k] = w[0][k];
#pragma unroll
      for (int r = 1; r < kMaxSplit; ++r)
        if (r < parts.split) v[k] += w[r][k];
    }
    T* out = static_cast<T*>(p.c) + (int64_t)(row0 + first + row) * p.ldc + col0 + col;
    if constexpr (kPull) {
      if (!__any_sync(0xFFFFFFFFu, aborted) && in) store8(out, v, min(8, ncols - col), p.c_unit);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (col + STEP * k < ncols) put(out + STEP * k, v[k]);
    }
  }
}

// T: the type of C; kWhole: its rows are whole 32-byte sectors. A kernel for
// each, since code for all in one leaves the epilogue's loop short of
// registers: 125.7 us against 109.1 at 4096 x 4096 x 7168 with three types.
template <typename T, bool kWhole>
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
  // STAGES: the stage's MMAs are done (one commit) and its factors are in
  // shared memory (the two scale warps). The epilogue waits for it before it
  // reads the products, the producer before it fills the stage again, a scale
  // warp before it writes the factors of STAGES blocks later. It cannot
  // complete again before the epilogue has seen it: that takes the MMAs of
  // STAGES blocks later, which wait for the epilogue's release of a buffer
  // that it gives only after this block. For the same reason the factors of
  // all but the last six blocks are used up when a barrier completes, and
  // eight slots need no barrier of their own.
  const uint32_t bar_done = bar_full + STAGES * 8;
  const uint32_t bar_acce = bar_done + STAGES * 8;      // 2: the epilogue has read buffer b, columns 256 b on
  const uint32_t bar_aux = bar_acce + 16;               // MMA drain on abort
  const uint32_t bar_never = bar_aux + 8;               // never arrived on (failure-path test)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_MISC + 4);
  InFlight* in_flight = reinterpret_cast<InFlight*>(smem + OFF_MISC + 16);
  float* scales = reinterpret_cast<float*>(smem + OFF_SCALE);
  int32_t* bounds = reinterpret_cast<int32_t*>(smem + OFF_SCHED);
  int32_t* tile_start = bounds + p.E + 1;
  const int E = p.E, NT = (p.N + BN - 1) / BN;

  load_bounds(p, bounds);
  if (tid == 32) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(bar_full + 8 * s, 1);
      mbar_init(bar_done + 8 * s, 3);
    }
    for (int b = 0; b < 2; ++b) mbar_init(bar_acce + 8 * b, 8);
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
  const Sched sch{bounds, tile_start, E, NT, p.N, BM, BN};
  if (warp == 0) scan_tiles(sch, bounds, tile_start);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int total = tile_start[E];
  const int KB = p.KB;
  // One CTA takes whole tiles in turn; a cluster of `split` takes one tile,
  // each CTA a range of the blocks of K.
  const int split = p.split;
  const int rank = split > 1 ? (int)cluster_ctarank() : 0;
  const int first = (int)blockIdx.x / split, stride = (int)gridDim.x / split;
  const int kb0 = KB * rank / split, kb1 = KB * (rank + 1) / split;

  if (warp == 0 && lane == 0) {
    // ---------------------------------------------------------------- producer
    // A weight tile read by one activation tile only is streamed (evict
    // first); one that several read keeps normal priority.
    const uint64_t pol_w1 = l2_policy_evict_first();
    const uint64_t pol_wn = l2_policy_evict_normal();
    const uint64_t pol_a = l2_policy_evict_last();
    uint32_t stage = 0, phase = 0, filled = 0, fill_phase = 0;
    bool ok = true;
    for (int t = first; ok && t < total; t += stride) {
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
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!wait_bounded(bar_done + 8 * stage, phase ^ 1, abort_flag, p.wait_limit_ns, p.status, 31)) {
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
    in_flight->filled = filled;
    in_flight->fill_phase = fill_phase;
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    // The whole warp runs the loop and one elected lane issues, so that the
    // descriptors stay in uniform registers.
    const bool leader = elect_one();
    uint32_t g = 0;
    bool ok = true, issued = false;
    const uint64_t adesc0 = sdesc_kmajor_sw128(sbase);
    const uint64_t bdesc0 = sdesc_kmajor_sw128(sbase + OFF_B);
    if (p.test_stall == 1 && first < total)
      ok = wait_warp(bar_never, 0, abort_flag, p.wait_limit_ns, p.status, 32);
    for (int t = first; ok && t < total; t += stride) {
      int e, nb, row0, rows, ncols;
      sch.decode(t, e, nb, row0, rows, ncols);
      const uint32_t idesc = idesc_e4m3(BM, (ncols + 15) / 16 * 16);
      for (int kb = kb0; kb < kb1; ++kb, ++g) {
        const uint32_t stage = g % STAGES, buf = g & 1u;
        ok = wait_warp(bar_full + 8 * stage, g / STAGES & 1u, abort_flag, p.wait_limit_ns, p.status, 34) &&
             wait_warp(bar_acce + 8 * buf, ((g >> 1) & 1u) ^ 1u, abort_flag, p.wait_limit_ns, p.status, 33);
        if (__builtin_expect(!ok, 0)) break;
        tc_fence_after();
        const uint64_t ad = adesc0 + ((stage * A_BYTES) >> 4);
        const uint64_t bd = bdesc0 + ((stage * B_BYTES) >> 4);
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < BK / 32; ++kk)   // 32 bytes of every row further per step
            tc_mma_f8(tmem + buf * BN, ad + 2 * kk, bd + 2 * kk, idesc, kk != 0 ? 1u : 0u);
          tc_commit(bar_done + 8 * stage);
        }
        issued = true;
      }
    }
    if (leader) in_flight->issued = issued;
  } else if (warp == 2 || warp == 3) {
    // ---------------------------------------------------------------- scales
    // Thread i makes the factors of rows i and i + 64 for both column halves
    // (a weight block each), up to four blocks ahead of the epilogue, which
    // then reads one word a block; the scales of the next four blocks are on
    // their way meanwhile. With the loads in the epilogue, every block waited
    // for them (linear 4096 x 4096 x 7168: 147 us against 114 with a constant
    // in their place).
    const int i = tid - 64;
    uint32_t g = 0;
    bool ok = p.test_stall != 2;
    for (int t = first; ok && t < total; t += stride) {
      int e, nb, row0, rows, ncols;
      sch.decode(t, e, nb, row0, rows, ncols);
      const float* sa = p.a_sf + (int64_t)row0 * KB;
      const float* sw0 = p.w_sf + ((int64_t)e * p.NB + nb * 2) * KB;
      const float* sw1 = ncols > HN ? sw0 + KB : sw0;
      float a0[4], a1[4], w0[4], w1[4];
      auto fetch = [&](int kg) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const bool in = kg + k < kb1;
          w0[k] = in ? __ldg(sw0 + kg + k) : 0.0f;
          w1[k] = in ? __ldg(sw1 + kg + k) : 0.0f;
          a0[k] = in && i < rows ? __ldg(sa + (int64_t)i * KB + kg + k) : 0.0f;
          a1[k] = in && i + 64 < rows ? __ldg(sa + (int64_t)(i + 64) * KB + kg + k) : 0.0f;
        }
      };
      fetch(kb0);
      for (int kg = kb0; ok && kg < kb1; kg += 4) {
        float f[4][4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          f[k][0] = a0[k] * w0[k];
          f[k][1] = a1[k] * w0[k];
          f[k][2] = a0[k] * w1[k];
          f[k][3] = a1[k] * w1[k];
        }
        fetch(kg + 4);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (kg + k < kb1) {
            const uint32_t bar = bar_done + 8 * (g % STAGES);
            ok = wait_warp(bar, (g / STAGES & 1u) ^ 1u, abort_flag, p.wait_limit_ns, p.status, 36);
            if (!ok) break;
            float* out = scales + (g % kScaleSlots) * (2 * BM) + i;
#pragma unroll
            for (int h = 0; h < 4; ++h) out[64 * h] = f[k][h];
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
            ++g;
          }
        }
      }
    }
  } else if (warp >= kEpiWarp0) {
    // ---------------------------------------------------------------- epilogue
    const int quad = warp & 3;              // TMEM lane quadrant this warp may access
    const int half = (warp - kEpiWarp0) >> 2;
    const int col0 = half * HN;             // its columns are those of one 128-wide weight block
    const int row = quad * 32 + lane;
    const uint32_t taddr = tmem + (static_cast<uint32_t>(quad * 32) << 16) + col0;
    uint32_t g = 0;
    bool ok = true;
    for (int t = first; ok && t < total; t += stride) {
      int e, nb, row0, rows, ncols;
      sch.decode(t, e, nb, row0, rows, ncols);
      const bool live = quad * 32 < rows && col0 < ncols;   // the whole warp
      float acc[HN];
#pragma unroll
      for (int i = 0; i < HN; ++i) acc[i] = 0.0f;
      for (int kb = kb0; kb < kb1; ++kb, ++g) {
        const uint32_t stage = g % STAGES, buf = g & 1u;
        ok = wait_warp(bar_done + 8 * stage, g / STAGES & 1u, abort_flag, p.wait_limit_ns, p.status, 35);
        if (__builtin_expect(!ok, 0)) break;
        tc_fence_after();
        const float s = scales[(g % kScaleSlots) * (2 * BM) + half * BM + row];
        if (live) {
#pragma unroll
          for (int c = 0; c < HN / 16; ++c) {
            uint32_t v[16];
            tc_ld16_wait(taddr + buf * BN + 16 * c, v);
            if (c + 1 == HN / 16) {   // all read: released before the last are added
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(bar_acce + 8 * buf);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[16 * c + i] = fmaf(__uint_as_float(v[i]), s, acc[16 * c + i]);
          }
        } else {
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_acce + 8 * buf);
        }
      }
      // (a cluster has one tile: its rings are free for the parts once all of
      // its CTAs' products are read)
      if (split > 1) cluster_sync_all();
      if (!ok || !live) continue;
      if (split > 1) {
        if (row < rows) {
          const Parts parts{sbase, kPartBytes, (rows + split - 1) / split, rank, split, 0};
          const uint32_t part = parts.slot(row) + col0 * 4;
#pragma unroll
          for (int i = 0; i < HN; i += 4) st_shared_cluster_v4(part + 4 * i, acc + i);
        }
        continue;
      }
      T* out = static_cast<T*>(p.c) + (int64_t)(row0 + quad * 32) * p.ldc + nb * BN + col0;
      const int n = min(HN, ncols - col0);
      if constexpr (kWhole) store_rows(out, p.ldc, acc, rows - quad * 32, n, lane);
      else if (row < rows) store_row_shifted(out + lane * p.ldc, acc, n);
    }
  }

  if (split > 1) {
    __syncwarp();
    if (warp < kEpiWarp0) cluster_sync_all();   // the epilogue's, above
    // every role of every CTA has ended: one that gave up tells the others
    if (tid < split && *abort_flag)
      st_shared_cluster_u32(mapa_shared(smem_addr(smem + OFF_MISC + 4), tid), 1u);
    __syncwarp();
    cluster_sync_all();                         // all parts are where they are joined
    int e, nb, row0, rows, ncols;
    sch.decode(first, e, nb, row0, rows, ncols);
    if (!*abort_flag)
      join_parts<T, BN, false>(p, Parts{sbase, kPartBytes, (rows + split - 1) / split, rank, split, 0}, row0, rows,
                               nb * BN, ncols, kThreads);
  }

  tc_fence_before();
  __syncthreads();
  if (warp < 2 && *abort_flag) drain(*in_flight, warp, lane, STAGES, bar_full, bar_aux);
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

// ------------------------------------------------------------------ few rows
//
// Tiles of at most NT activation rows (16, 32 or 64) x 128 weight rows, with
// the operands exchanged: the weight rows are the MMA's M, the activation rows
// its N, so that a lane holds one weight row and a block's products are NT
// columns instead of 256. Reading them back costs NT / 256 of the time, four
// buffers hide the hand-offs, and a tile of half the weight rows gives twice
// the CTAs: with few rows the product is a stream of the weights from HBM, and
// what counts is that every SM keeps loads in flight. One unit of work is one
// tile and one range of its blocks of K (a cluster of `split` CTAs shares a
// tile); a stage is small enough for two CTAs on an SM (for 16 rows with up to
// 343 groups), so that one unit's loads run under another's beginning and end
// (8 rows of 256 groups, 4096 x 7168: 41.2 us; one CTA 47.7). The sums leave
// through shared memory, since a lane holds a column of C, joined over the
// cluster.
// Warp roles (256 threads): 0 producer, 1 MMA, 2 factors, 4-7 epilogue. (Eight
// epilogue warps for 64 rows measured the same: 14.5 us against 14.3 at
// 64 x 4096 x 7168.)
template <int NT>
struct Few {
  static constexpr int STAGES = NT == 16 ? 6 : NT == 32 ? 5 : 4;
  static constexpr int BUFS = 4;             // at most STAGES (see bar_done)
  static constexpr int W_BYTES = 128 * BK;   // 16 KB
  static constexpr int T_BYTES = NT * BK;
  static constexpr int OFF_T = STAGES * W_BYTES;
  static constexpr int OFF_BAR = OFF_T + STAGES * T_BYTES;
  // factors change hands four blocks at a time, four such groups on their way
  static constexpr int SBLOCKS = 4, SSLOTS = 4;
  static constexpr int SCALE_FLOATS = SBLOCKS * NT;        // [block][row]
  static constexpr int OFF_SCALE = OFF_BAR + 256;
  static constexpr int OFF_MISC = OFF_SCALE + SSLOTS * SCALE_FLOATS * 4;
  static constexpr int OFF_SCHED = OFF_MISC + 64;
  static constexpr int PART_BYTES = 128 * 4 + 16;          // a row of partial sums
  static constexpr uint32_t TMEM = BUFS * NT;
  static_assert(NT * PART_BYTES <= OFF_BAR, "the partial sums lie in the ring");
  static_assert(BUFS <= STAGES, "a barrier of a stage would complete twice unseen");
  static_assert(2 * (shared_bytes(OFF_SCHED, 256) + 1024) <= kSharedOfSM, "two CTAs on an SM");
};

constexpr int kFewThreads = 256;

template <int NT>
__global__ void __launch_bounds__(kFewThreads, 2)
    fp8_gemm_few_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_w,
                        const Params p) {
  using C = Few<NT>;
  constexpr int STAGES = C::STAGES, BUFS = C::BUFS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sbase = smem_addr(smem);
  const uint32_t bar_full = sbase + C::OFF_BAR;         // STAGES: a stage's tiles landed
  const uint32_t bar_done = bar_full + STAGES * 8;      // STAGES: its MMAs are done (as in fp8_gemm_kernel)
  const uint32_t bar_acce = bar_done + STAGES * 8;      // BUFS: the epilogue has read a buffer
  const uint32_t bar_sff = bar_acce + BUFS * 8;         // SSLOTS: a group of factors is in shared memory
  const uint32_t bar_sfe = bar_sff + C::SSLOTS * 8;   // SSLOTS: the epilogue has used it
  const uint32_t bar_aux = bar_sfe + C::SSLOTS * 8;   // MMA drain on abort
  const uint32_t bar_never = bar_aux + 8;               // never arrived on (failure-path test)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  InFlight* in_flight = reinterpret_cast<InFlight*>(smem + C::OFF_MISC + 16);
  float* scales = reinterpret_cast<float*>(smem + C::OFF_SCALE);
  int32_t* bounds = reinterpret_cast<int32_t*>(smem + C::OFF_SCHED);
  int32_t* tile_start = bounds + p.E + 1;
  const Sched sch{bounds, tile_start, p.E, p.NB, p.N, NT, 128};

  const int split = p.split;
  const int rank = split > 1 ? (int)cluster_ctarank() : 0;
  const int unit = (int)blockIdx.x / split;
  int e = 0, nb = 0, row0 = 0, rows = 0, ncols = 0, kb0 = 0, kb1 = 0;
  auto blocks_of_k = [&]() {
    kb0 = p.KB * rank / split;
    kb1 = p.KB * (rank + 1) / split;
  };
  if (!p.offsets) {   // one group: the tile needs no schedule
    const int mt = (p.M + NT - 1) / NT;
    nb = unit / mt;
    row0 = (unit - nb * mt) * NT;
    rows = min(NT, p.M - row0);
    ncols = min(128, p.N - nb * 128);
    blocks_of_k();
  } else {
    load_bounds(p, bounds);
  }
  // the producer's state (thread 0)
  uint32_t p_stage = 0, p_phase = 0, filled = 0, fill_phase = 0;
  int p_kb = kb0;
  auto fill = [&]() {   // the next block of K into the next stage
    const uint32_t full = bar_full + 8 * p_stage;
    mbar_arrive_expect_tx(full, C::W_BYTES + C::T_BYTES);
    tma_load_2d(sbase + p_stage * C::W_BYTES, &tm_w, full, p_kb * BK, e * p.N + nb * 128,
                p.w_once ? l2_policy_evict_first() : l2_policy_evict_normal());
    tma_load_2d(sbase + C::OFF_T + p_stage * C::T_BYTES, &tm_a, full, p_kb * BK, row0, l2_policy_evict_last());
    filled |= 1u << p_stage;
    fill_phase = (fill_phase & ~(1u << p_stage)) | (p_phase << p_stage);
    ++p_kb;
    if (++p_stage == STAGES) {
      p_stage = 0;
      p_phase ^= 1;
    }
  };
  if (tid == 0) {
    prefetch_tensormap(&tm_w);
    prefetch_tensormap(&tm_a);
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(bar_full + 8 * s, 1);
      mbar_init(bar_done + 8 * s, 1);
    }
    for (int b = 0; b < BUFS; ++b) mbar_init(bar_acce + 8 * b, 4);
    for (int b = 0; b < C::SSLOTS; ++b) {
      mbar_init(bar_sff + 8 * b, 32);
      mbar_init(bar_sfe + 8 * b, 4);
    }
    mbar_init(bar_aux, 1);
    mbar_init(bar_never, 1);
    *abort_flag = 0;
    fence_mbar_init();
    // one group: the first loads are on their way while the rest is set up
    for (int i = 0; i < STAGES && p_kb < kb1; ++i) fill();
  }
  if (warp == 1) {
    __syncwarp();
    tmem_alloc(smem_addr(tmem_slot), C::TMEM);
    tmem_relinquish();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (p.offsets) {
    if (warp == 0) scan_tiles_by_runs(sch, bounds, tile_start);
    __syncthreads();
    if (unit < tile_start[p.E]) {   // the same for every CTA of a cluster
      sch.decode(unit, e, nb, row0, rows, ncols);
      blocks_of_k();
      p_kb = kb0;
    }
  }
  const bool any = rows > 0;

  if (warp == 0 && lane == 0) {
    // ---------------------------------------------------------------- producer
    bool ok = true;
    while (ok && p_kb < kb1) {
      ok = wait_bounded(bar_done + 8 * p_stage, p_phase ^ 1, abort_flag, p.wait_limit_ns, p.status, 41);
      if (ok) fill();
    }
    in_flight->filled = filled;
    in_flight->fill_phase = fill_phase;
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    const bool leader = elect_one();
    uint32_t stage = 0, phase = 0, buf = 0, bphase = 1;
    bool ok = true, issued = false;
    const uint64_t wdesc0 = sdesc_kmajor_sw128(sbase);
    const uint64_t tdesc0 = sdesc_kmajor_sw128(sbase + C::OFF_T);
    if (p.test_stall == 1 && any)
      ok = wait_warp(bar_never, 0, abort_flag, p.wait_limit_ns, p.status, 42);
    for (int kb = kb0; ok && kb < kb1; ++kb) {
      ok = wait_warp(bar_acce + 8 * buf, bphase, abort_flag, p.wait_limit_ns, p.status, 43) &&
           wait_warp(bar_full + 8 * stage, phase, abort_flag, p.wait_limit_ns, p.status, 44);
      if (!ok) break;
      tc_fence_after();
      const uint64_t wd = wdesc0 + ((stage * C::W_BYTES) >> 4);
      const uint64_t td = tdesc0 + ((stage * C::T_BYTES) >> 4);
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < BK / 32; ++kk)
          tc_mma_f8(tmem + buf * NT, wd + 2 * kk, td + 2 * kk, idesc_e4m3(128, NT), kk != 0 ? 1u : 0u);
        tc_commit(bar_done + 8 * stage);
      }
      issued = true;
      if (++stage == STAGES) {
        stage = 0;
        phase ^= 1;
      }
      if (++buf == BUFS) {
        buf = 0;
        bphase ^= 1;
      }
    }
    if (leader) in_flight->issued = issued;
  } else if (warp == 2) {
    // ---------------------------------------------------------------- factors
    constexpr int R = (NT + 31) / 32;      // activation rows of a lane
    uint32_t slot = 0, phase = 0;
    const bool ok = p.test_stall != 2;
    const float* sa = p.a_sf + (int64_t)row0 * p.KB;
    const float* sw = p.w_sf + ((int64_t)e * p.NB + nb) * p.KB;
    for (int kg = kb0; ok && kg < kb1; kg += C::SBLOCKS) {
      float a[R][C::SBLOCKS];
#pragma unroll
      for (int k = 0; k < C::SBLOCKS; ++k) {
        const bool in = kg + k < kb1;
        const float w = in ? __ldg(sw + kg + k) : 0.0f;
#pragma unroll
        for (int h = 0; h < R; ++h) {
          const int r = lane + 32 * h;
          a[h][k] = in && r < rows ? __ldg(sa + (int64_t)r * p.KB + kg + k) * w : 0.0f;
        }
      }
      if (!wait_warp(bar_sfe + 8 * slot, phase ^ 1, abort_flag, p.wait_limit_ns, p.status, 46)) break;
#pragma unroll
      for (int k = 0; k < C::SBLOCKS; ++k)
#pragma unroll
        for (int h = 0; h < R; ++h)
          if (lane + 32 * h < NT) scales[slot * C::SCALE_FLOATS + k * NT + lane + 32 * h] = a[h][k];
      mbar_arrive(bar_sff + 8 * slot);
      if (++slot == C::SSLOTS) {
        slot = 0;
        phase ^= 1;
      }
    }
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- epilogue
    const int quad = warp & 3;
    const uint32_t taddr = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    uint32_t stage = 0, phase = 0, buf = 0, slot = 0, sphase = 0;
    bool ok = true;
    float acc[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[i] = 0.0f;
    for (int kb = kb0; kb < kb1; ++kb) {
      const int in_group = (kb - kb0) % C::SBLOCKS;
      if (in_group == 0)
        ok = wait_warp(bar_sff + 8 * slot, sphase, abort_flag, p.wait_limit_ns, p.status, 47);
      ok = ok && wait_warp(bar_done + 8 * stage, phase, abort_flag, p.wait_limit_ns, p.status, 45);
      if (!ok) break;
      tc_fence_after();
      const float4* f = reinterpret_cast<const float4*>(scales + slot * C::SCALE_FLOATS + in_group * NT);
#pragma unroll
      for (int c = 0; c < NT / 16; ++c) {
        if (16 * c < rows) {
          uint32_t v[16];
          tc_ld16_wait(taddr + buf * NT + 16 * c, v);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float4 s = f[4 * c + q];
            acc[16 * c + 4 * q] = fmaf(__uint_as_float(v[4 * q]), s.x, acc[16 * c + 4 * q]);
            acc[16 * c + 4 * q + 1] = fmaf(__uint_as_float(v[4 * q + 1]), s.y, acc[16 * c + 4 * q + 1]);
            acc[16 * c + 4 * q + 2] = fmaf(__uint_as_float(v[4 * q + 2]), s.z, acc[16 * c + 4 * q + 2]);
            acc[16 * c + 4 * q + 3] = fmaf(__uint_as_float(v[4 * q + 3]), s.w, acc[16 * c + 4 * q + 3]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_acce + 8 * buf);
      if (in_group == C::SBLOCKS - 1 || kb + 1 == kb1) {
        if (lane == 0) mbar_arrive(bar_sfe + 8 * slot);
        if (++slot == C::SSLOTS) {
          slot = 0;
          sphase ^= 1;
        }
      }
      if (++stage == STAGES) {
        stage = 0;
        phase ^= 1;
      }
      if (++buf == BUFS) buf = 0;
    }
    // every MMA of this CTA is done and its operands are read: the ring is free
    if (ok) {
#pragma unroll
      for (int i = 0; i < NT; ++i)
        if (i < rows) *reinterpret_cast<float*>(smem + i * C::PART_BYTES + (quad * 32 + lane) * 4) = acc[i];
    }
  }

  __syncwarp();
  if (split > 1) cluster_sync_all();
  else __syncthreads();
  const bool gave_up = *abort_flag != 0;   // all roles have ended
  const Parts parts{sbase, C::PART_BYTES, rows > split ? (rows + split - 1) / split : 1, rank, split,
                    smem_addr(smem + C::OFF_MISC + 4)};
  auto join = [&](auto type) {
    using T = decltype(type);
    if (split > 1) join_parts<T, 128, true>(p, parts, row0, rows, nb * 128, ncols, kFewThreads);
    else join_parts<T, 128, false>(p, parts, row0, rows, nb * 128, ncols, kFewThreads);
  };
  if (!gave_up) {
    if (p.c_type == NVFP4MOE_BF16) join(__nv_bfloat16());
    else if (p.c_type == NVFP4MOE_F16) join(__half());
    else join(0.0f);
  }
  __syncwarp();
  if (split > 1) cluster_sync_all();   // every CTA's part stays until all have read it
  tc_fence_before();
  __syncthreads();
  if (gave_up && warp < 2) drain(*in_flight, warp, lane, STAGES, bar_full, bar_aux);
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM);
  }
}

constexpr int kMaxDevices = 64;

// Lets a kernel take the shared memory of kMaxGroups groups, once per device
// (index: one per kernel). The limit is the function's, not a launch's: set to
// what each call needs, another thread's call could lower it before the launch.
template <typename Kernel>
bool allow_shared(Kernel kernel, int index, size_t most) {
  static std::atomic<bool> known[kMaxDevices][9];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return false;
  std::atomic<bool>& set = known[dev][index];
  if (set.load(std::memory_order_acquire)) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  set.store(true, std::memory_order_release);
  return true;
}

// Clusters of `split` CTAs of a kernel that fit the device at once, asked once
// per device (index: one per kernel), with the shared memory of kMaxGroups
// groups: the answer, and with it the order of a product's sums, is the same
// whatever was called before. (It counts one CTA to an SM for every kernel
// that allocates tensor memory, also where two do run on one.)
template <typename Kernel>
int resident_clusters(Kernel kernel, int index, int threads, size_t most, int split) {
  static std::atomic<int> known[kMaxDevices][4][3];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  std::atomic<int>& slot = known[dev][index][split == 2 ? 0 : split == 4 ? 1 : 2];
  int n = slot.load(std::memory_order_relaxed);
  if (n == 0) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)split, 1, 1);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = most;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
      cudaGetLastError();
      return 0;   // (not kept: another call may be answered)
    }
    if (n <= 0) n = -1;
    slot.store(n, std::memory_order_relaxed);
  }
  return n;
}

template <typename Kernel, typename... Args>
int launch_clusters(Kernel kernel, int64_t grid, int threads, size_t smem, int split, void* stream,
                    const Args&... args) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)grid, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = as_stream(stream);
  cfg.attrs = attr;
  cfg.numAttrs = split > 1 ? 1 : 0;
  cudaLaunchKernelEx(&cfg, kernel, args...);
  return launch_status();
}

// How a kernel would run a product, and the time estimated for it.
struct Plan {
  int split = 1;   // CTAs (a cluster) to a tile
  float us = 0;
};

// Where there are few tiles, each goes to a cluster of 2, 4 or 8 CTAs that
// share its blocks of K, if all clusters run at once and it is estimated to be
// faster. A CTA takes `block` us a block of K; joining the parts takes 0.5 us and
// join[0 .. 2] us a row of the tile with 2, 4 and 8 CTAs (distributed shared
// memory moves about 10 bytes a cycle and SM). Measured, split 1 / 2 / 4 / 8 of the 128-row tiles: 128 x 512 x
// 2048 12.0 / 12.7 / 12.6 / 12.8 us, 128 x 4096 x 7168 27.6 / 20.7 / 16.9, 1 x
// 4096 x 7168 26.1 / 16.3 / 11.0 (15 clusters of 8 fit, and 16 would be needed).
struct Costs {
  float block, join[3], fixed;
};

template <typename Resident>
Plan plan(int64_t units, int KB, int rows, const Costs& c, int sms, Resident resident) {
  Plan best;
  for (int split = 1; split <= kMaxSplit && split <= KB; split *= 2) {
    if (split > 1 && units > resident(split)) break;
    const float waves = units * split > sms ? (float)units * split / sms : 1.0f;
    float us = c.block * ((KB + split - 1) / split) * waves + c.fixed;
    if (split > 1) us += 0.5f + c.join[split == 2 ? 0 : split == 4 ? 1 : 2] * rows;
    if (split == 1 || us < best.us) best = Plan{split, us};
  }
  return best;
}

// Activation tiles of tm rows, at most.
int64_t tiles_of(const Params& p, int tm) {
  if (!p.offsets) return ceil_div(p.M, tm);
  return p.M / tm + (p.E < p.M ? p.E : p.M);
}

template <int NT>
struct FewLaunch {
  size_t smem;
  int64_t units;
  Plan plan;
  bool ok;
  FewLaunch(const Params& p, int sms) {
    smem = shared_bytes(Few<NT>::OFF_SCHED, p.E);
    units = tiles_of(p, NT) * p.NB;
    const size_t most = shared_bytes(Few<NT>::OFF_SCHED, kMaxGroups);
    ok = units * kMaxSplit < (1ll << 31) && allow_shared(fp8_gemm_few_kernel<NT>, NT == 16 ? 6 : NT == 32 ? 7 : 8, most);
    if (!ok) return;
    // a block: split 1 of 56 blocks takes 16.4, 18.8 and 29.1 us
    const Costs costs{NT == 16 ? 0.22f : NT == 32 ? 0.26f : 0.5f, {0.013f, 0.022f, 0.037f}, 4.0f};
    plan = nvfp4moe::plan(units, p.KB, p.M < NT ? p.M : NT, costs, sms, [&](int split) {
      return resident_clusters(fp8_gemm_few_kernel<NT>, NT == 16 ? 1 : NT == 32 ? 2 : 3, kFewThreads, most, split);
    });
  }
  int run(const uint8_t* a_codes, int64_t lda, const uint8_t* w_codes, int64_t ldw, Params& p, void* stream) const {
    CUtensorMap ma, mw;
    if (!make_codes_map(&ma, a_codes, p.M, p.K, lda, NT) ||
        !make_codes_map(&mw, w_codes, (int64_t)p.E * p.N, p.K, ldw, 128))
      return NVFP4MOE_ERR_INVALID;
    p.w_once = !p.offsets && p.M <= NT;
    p.split = plan.split;
    return launch_clusters(fp8_gemm_few_kernel<NT>, units * p.split, kFewThreads, smem, p.split, stream, ma, mw, p);
  }
};

int launch(const uint8_t* a_codes, int64_t lda, const uint8_t* w_codes, int64_t ldw, Params& p, void* stream) {
  p.status = device_status_word();
  NVFP4_CHECK(p.status, NVFP4MOE_ERR_LAUNCH);
  p.wait_limit_ns = wait_limit_ns();
  p.test_stall = test_stall_on();
  const int sms = device_num_sms();
  NVFP4_CHECK(sms > 0, NVFP4MOE_ERR_LAUNCH);
  auto kernel = p.c_type == NVFP4MOE_BF16
                    ? (p.c_32B ? fp8_gemm_kernel<__nv_bfloat16, true> : fp8_gemm_kernel<__nv_bfloat16, false>)
                : p.c_type == NVFP4MOE_F16 ? (p.c_32B ? fp8_gemm_kernel<__half, true> : fp8_gemm_kernel<__half, false>)
                                           : (p.c_32B ? fp8_gemm_kernel<float, true> : fp8_gemm_kernel<float, false>);
  const size_t smem = shared_bytes(OFF_SCHED, p.E);
  const int index = 2 * (p.c_type == NVFP4MOE_BF16 ? 0 : p.c_type == NVFP4MOE_F16 ? 1 : 2) + (p.c_32B ? 1 : 0);
  const size_t most = shared_bytes(OFF_SCHED, kMaxGroups);
  if (!allow_shared(kernel, index, most)) return NVFP4MOE_ERR_LAUNCH;
  const int64_t units = tiles_of(p, BM) * ceil_div(p.N, BN);
  // (groups: the number of tiles is only known on the device; this kernel's
  // CTAs then take them in turn)
  const Costs costs{0.39f, {0.026f, 0.038f, 0.043f}, 6.0f};
  Plan tiles = plan(units, p.KB, p.M < BM ? p.M : BM, costs, sms, [&](int split) {
    return p.offsets ? 0 : resident_clusters(kernel, 0, kThreads, most, split);
  });
  // Few rows: the other kernel where it is estimated to be faster (64 x 4096 x
  // 7168 13.2 us against 16.9, 64 x 16384 x 7168 32.7 against 24.2). Rows of a
  // group: the mean of the groups that can have one, and room for twice that.
  const int rows = p.offsets ? 2 * (int)ceil_div(p.M, p.E < p.M ? p.E : p.M) : p.M;
  if (rows <= 16) {
    const FewLaunch<16> f(p, sms);
    if (f.ok && f.plan.us <= tiles.us) return f.run(a_codes, lda, w_codes, ldw, p, stream);
  } else if (rows <= 32) {
    const FewLaunch<32> f(p, sms);
    if (f.ok && f.plan.us <= tiles.us) return f.run(a_codes, lda, w_codes, ldw, p, stream);
  } else if (tiles_of(p, 64) * p.NB <= 4 * sms) {
    const FewLaunch<64> f(p, sms);
    if (f.ok && f.plan.us <= tiles.us) return f.run(a_codes, lda, w_codes, ldw, p, stream);
  }
  // Rows that do not start on 128-byte lines make two line requests a block of
  // K each, and 256 bytes fetched into L2 for each are too many where tiles are
  // read again from there: 4096 x 4864 x 2000 55.1 us with 128 bytes, 62.6 with
  // 256. Weights that are read once, as where the groups have less than a tile of
  // rows, stay with 256: 64 groups of 64 rows, 4096 x 2000, 94.0 us against 97.6.
  auto line = [](const void* base, int64_t ld, bool again) {
    return again && !(aligned(base, 128) && ld % 128 == 0) ? 128 : 256;
  };
  const bool w_again = p.M >= (int64_t)BM * p.E;
  CUtensorMap ma[4], mb[2];
  const int boxes[4] = {16, 32, 64, 128};
  for (int i = 0; i < 4; ++i)
    if (!make_codes_map(&ma[i], a_codes, p.M, p.K, lda, boxes[i], line(a_codes, lda, true))) return NVFP4MOE_ERR_INVALID;
  for (int i = 0; i < 2; ++i)
    if (!make_codes_map(&mb[i], w_codes, (int64_t)p.E * p.N, p.K, ldw, 128 << i, line(w_codes, ldw, w_again)))
      return NVFP4MOE_ERR_INVALID;
  p.split = tiles.split;
  const int64_t grid = p.split > 1 ? units * p.split : units < sms ? units : sms;
  return launch_clusters(kernel, grid, kThreads, smem, p.split, stream, ma[0], ma[1], ma[2], ma[3], mb[0],
                         mb[1], p);
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
  p.c_unit = 16;
  while (p.c_unit > es && !(aligned(c, p.c_unit) && ldc * es % p.c_unit == 0 && N * es % p.c_unit == 0)) p.c_unit /= 2;
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
