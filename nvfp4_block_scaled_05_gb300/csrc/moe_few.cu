// An expert layer for a few tokens (at most 32) with 8-bit block-scaled weights,
// in two kernels:
//   1. top-k softmax routing; h = silu(x Wg^T) * (x Wu^T) for every token and each
//      of its experts
//   2. out = h Wd^T; y = sum over a token's experts of weight * out, plus the
//      residual
// With few tokens the layer is one pass over the weights of the experts that
// have a token, so activations are not rounded to 8 bits: that would save
// nothing. Products are mma.sync of f16 operands with f32 sums: E4M3 codes are
// f16 numbers, and tcgen05 has no form that takes 8-bit weights with wider
// activations. 16 weight rows are the MMA's M, 8 tokens its N. The loop moves its
// codes at up to 6.7 TB/s, which is HBM's rate. An expert's tokens beyond 8 are
// another entry, which reads and converts the weights again. (With h of a BF16 result
// as one f16, see below, entries of 16, whose registers leave 8 warps, were slower at
// every load measured: 91 against 83 us for 32 tokens of 2 of 16 experts 4096/2048,
// and 171 against 140 where each token takes all of 8; the entries of an expert side
// by side in time, for L2's sake, 162; one copy for both tiles of a unit, or refilled
// as soon as it is read, the same.)
//
// A row's activations are taken in the weights' blocks of 128: each block is
// scaled by a power of two that brings its largest magnitude to [2^14, 2^15),
// and is held as one f16 or as the sum of two. One holds BF16 and F16 inputs
// exactly (every element above 2^-28 of its block's largest); F32 inputs and h,
// which is f32, take two, 22 bits, whatever y's type: with one, 11 bits, the sum
// carried an error that a BF16 y shows where a residual cancels most of it, and y
// differed from that of f32 sums by 4.9e-4 of its RMS, now by 6e-5. The second part
// takes 2 us of the 68 for one token of 256 experts 7168/2048, 15 of the 150 to 161
// for 32 tokens that each take all of 8 experts 4096/2048. The block's sums are
// scaled back with the weights' scale, in f32, and added in f32 in ascending order.
//
// Work: a unit is two tiles of 16 weight rows over the whole K (gate and up rows
// of the same columns of h, so that one lane holds both; or neighbouring rows of
// Wd). A block takes an equal run of the units, and its warps share the run's
// blocks of K evenly. Each warp streams its codes through a ring of its own in
// shared memory, filled by TMA, so that nothing waits for other warps; the run's
// activations lie in shared memory: those of all tokens or slots where they fit,
// else those of the experts at hand, else (a few tokens of one expert with a very
// wide K) two units a warp at a time go over K in pieces that do.
//
// The second kernel is launched with programmatic serialization: its blocks start
// as the first's end, route and fill their rings, then wait for the first's last.
// If the h of all slots fits, a block has all experts of its columns and makes y
// itself. Otherwise units are ordered by expert, out goes to the workspace in f32,
// and the last unit to finish for 32 columns (a counter, zeroed by the first
// kernel) adds up the token's experts in their order: the same result whichever
// it is.
//
// Every wait is bounded: one that exceeds the limit sets the device status word
// and ends the layer without a result; a warp that gave up waits for its copies.
//
// Measured in BF16, experts' K/I, with the fraction that reading the codes once
// takes at 6.79 TB/s: 32 tokens of 8 of 256 experts 7168/2048 1061 to 1076 us (98%),
// 16 of 128 550 us (96%), four of 64 185 us (90%), one of 256 68 us (76%); one token
// of 2 of 8 experts 128/128 9.3 us, which is two launches, two routings and the
// hand-over of h: what bounds every small layer. Where experts have more than 8
// tokens their entries do: 32 tokens of 2 of 8 experts 4096/2048 take 69 to 71 us
// (42%). fp8_moe_forward, with activations of 8 bits, takes 52 there, 77 for one
// token and 1004 for 32 of 256 experts 7168/2048.
#include "fp8_rows.cuh"

namespace nvfp4moe {
namespace {

constexpr int kMaxTokens = NVFP4MOE_FEW_TOKENS_MAX;
constexpr int kMaxSlots = kMaxTokens * 16;
static_assert(kMaxTokens <= 32, "a token is a bit of a word");
constexpr int kTileBytes = 2048;    // 16 rows x 128 codes
constexpr int kStageBytes = 2 * kTileBytes;
constexpr int kBlock = 128;
constexpr int kEntry = 8;           // tokens of an entry
// 96 KB of codes are on their way to an SM. Time in BF16, us, of one and of 32 tokens
// of 8 of 256 experts 7168/2048, of 32 tokens of 2 of 8 experts 4096/2048, and of all
// 8: 12 warps with 2 stages 69.1, 1127, 71 and 164; 12 with 3 68.9, 1136, 98 and 200;
// 16 with 2 72.5, 1179, 116 and 256; 10 with 3 71.8, 1115, 70 and 179; 8 with 4 70.4,
// 1270, 77 and 172 (the others have less room for activations, fewer warps, or
// both). One token of 2 of 8 experts 4096/2048 21.3 to 22.6, 4 of 6 of 64 experts
// 2048/512 in F16 28.0 to 30.2 with all of them.
constexpr int kWarps = 12, kStages = 2;

__device__ __forceinline__ void cp_async_4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// Quotients by a number that the host knows: a product's high half is at most one
// too large for numerators below 2^27 (the compiler's division takes 20 to 30
// dependent instructions, and each warp needs several before its first copy).
struct Divisor {
  uint32_t d, m;
  Divisor() = default;
  explicit Divisor(uint32_t by) : d(by), m(by == 1 ? 0xFFFFFFFFu : (uint32_t)(((1ull << 32) + by - 1) / by)) {}
};
__device__ __forceinline__ int operator/(int n, const Divisor& by) {
  const int q = (int)__umulhi((uint32_t)n, by.m);
  const int r = n - q * (int)by.d;
  return r < 0 ? q - 1 : r >= (int)by.d ? q + 1 : q;
}

// The routing of all tokens, in shared memory: both kernels' blocks make it
// themselves, the second's while the first's last blocks run.
struct Route {
  float weight[kMaxSlots];           // (T, k)
  uint16_t expert[kMaxSlots + 2];    // entries: experts that have a token, ascending
  uint16_t start[kMaxSlots + 2];     // their first places in slot[]
  uint16_t slot[kMaxSlots];          // t * k + j, by expert, then token
  uint8_t token[kMaxSlots];          // t
  int n;                             // entries
  int gave_up;                       // a wait ran out
  uint64_t never;                    // a barrier that nothing arrives on (failure-path test)
  uint64_t pad;
};
static_assert(sizeof(Route) % 16 == 0, "what follows is 16-byte aligned");

// A block's shared memory: the rings, parts of sums, the routing, barriers and
// scales, activations.
constexpr int kSmemBytes = 222 * 1024;
constexpr int kRowsBytes =
    (kSmemBytes - (int)sizeof(Route) - kWarps * (kStages * (kStageBytes + 16) + 4 * 512)) / 16 * 16;
static_assert(kRowsBytes >= kEntry * (2 * 256 + 4 + 16), "a block of an entry in two parts");
static_assert(kWarps * kStages * kStageBytes >= 1024 * 6 + 4 * kWarps, "the routing's scratch");

struct FewArgs {
  const void* src;          // rows of activations: x (a row a token) or h (a row a slot)
  int64_t lds;
  const float* logits;      // (T, E)
  int T, E, k;
  int width, KB;            // of a row; its blocks
  const float* sf;          // scales, (E, row_blocks, KB)
  int64_t rows, row_blocks; // weight rows of an expert
  int tiles, upe;           // tiles of 16 rows (of which half are gate rows), units of an expert
  Divisor by_upe, by_KB, by_k;
  float* dst;               // h or out
  int64_t ldd;
  int* counters;            // one for 32 output columns, then whether the first kernel gave up; it zeroes them
  int n_counters;           // without the last
  int resident;             // the activations of all tokens (slots) fit
  void* y;
  const void* residual;
  int64_t ldy, ldr;
  uint64_t wait_limit_ns;
  int* status;
  int test_stall;           // test hook: the first wait is for a barrier that nothing arrives on
};

// A converged warp's wait on a barrier, as wait_bounded; the result is the same in
// all lanes.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int* abort_flag, uint64_t limit_ns,
                                          int* status, int site) {
  if (__builtin_expect(__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity)), 1)) return true;
  return __all_sync(0xFFFFFFFFu, wait_bounded(bar, parity, abort_flag, limit_ns, status, site));
}

// Four E4M3 codes as four f16 (exact).
__device__ __forceinline__ void codes_to_f16(uint32_t four, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(four));
}

// d = a b + c.
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1,
                                        const float (&c)[4]) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

// route_token's result with fewer steps: logits as integers of the same order, so
// that a round is two reductions over the warp (the largest, then the lowest
// expert that has it) in place of ten shuffles.
template <int V>
__device__ __forceinline__ void route_token_fast(const float* __restrict__ row, int E, int k, int lane, int& my_i,
                                                 float& my_w) {
  uint32_t key[V];   // 0: no expert, or taken
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + 32 * i;
    float v = e < E ? row[e] : 0.0f;
    v = v == v ? v + 0.0f : -INFINITY;   // (one zero; a NaN ranks with -inf)
    const uint32_t u = __float_as_uint(v);
    key[i] = e < E ? ((u >> 31) ? ~u : u | 0x80000000u) : 0u;
  }
  uint32_t my_key = 0;
  my_i = 0;
  for (int j = 0; j < k; ++j) {
    uint32_t m = key[0];
#pragma unroll
    for (int i = 1; i < V; ++i) m = max(m, key[i]);
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    uint32_t e = 0xFFFFFFFFu;
#pragma unroll
    for (int i = V - 1; i >= 0; --i) e = key[i] == m ? (uint32_t)(lane + 32 * i) : e;
    e = __reduce_min_sync(0xFFFFFFFFu, e);
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = e == (uint32_t)(lane + 32 * i) ? 0u : key[i];
    if (lane == j) {
      my_key = m;
      my_i = (int)e;
    }
  }
  const float my_v = __uint_as_float((my_key >> 31) ? my_key & 0x7FFFFFFFu : ~my_key);
  const float vmax = __shfl_sync(0xFFFFFFFFu, my_v, 0);
  const float ex = lane < k ? expf(my_v - vmax) : 0.0f;
  float den = ex;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xFFFFFFFFu, den, o);
  my_w = ex / den;
}

// All tokens routed (moe_route_topk's rule), and the slots in expert order, an
// entry for each kEntry tokens of an expert. mask: E words, E half words and a
// word a warp of scratch. `meanwhile` is called by the warps without a
// token.
template <typename Meanwhile>
__device__ __forceinline__ void route_all(const FewArgs& a, Route& r, uint32_t* mask, Meanwhile meanwhile) {
  constexpr int kThreads = 32 * kWarps;
  constexpr int kMine = (kMaxSlots + kThreads - 1) / kThreads, kOwn = (1024 + kThreads - 1) / kThreads;
  int* totals = reinterpret_cast<int*>(mask + a.E);
  uint16_t* index = reinterpret_cast<uint16_t*>(totals + kWarps);
  uint16_t* ids = r.slot;   // (T, k), until the slots take the place
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto route = [&](int t, int& id, float& w) {
    const float* row = a.logits + (int64_t)t * a.E;
    if (a.E <= 64) route_token_fast<2>(row, a.E, a.k, lane, id, w);
    else if (a.E <= 256) route_token_fast<8>(row, a.E, a.k, lane, id, w);
    else route_token_fast<32>(row, a.E, a.k, lane, id, w);
  };
  if (a.T == 1) {   // each of the token's experts is an entry: one warp orders them
    if (warp == 0) {
      int id, at = 0;
      float w;
      route(0, id, w);
      for (int j = 0; j < a.k; ++j) at += __shfl_sync(0xFFFFFFFFu, id, j) < id;
      if (lane < a.k) {
        r.weight[lane] = w;
        r.expert[at] = (uint16_t)id;
        r.start[at] = (uint16_t)at;
        r.slot[at] = (uint16_t)lane;
        r.token[at] = 0;
      }
      if (lane == 0) {
        r.n = a.k;
        r.start[a.k] = (uint16_t)a.k;
      }
    } else {
      meanwhile();
    }
    __syncthreads();
    return;
  }
  for (int e = tid; e < a.E; e += kThreads) mask[e] = 0;
  __syncthreads();
  for (int t = warp; t < a.T; t += kWarps) {
    int id;
    float w;
    route(t, id, w);
    if (lane < a.k) {
      ids[t * a.k + lane] = (uint16_t)id;
      r.weight[t * a.k + lane] = w;
      atomicOr(&mask[id], 1u << t);
    }
  }
  if (warp >= a.T) meanwhile();
  __syncthreads();
  const int slots = a.T * a.k;
  uint16_t mine[kMine];
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int f = tid + i * kThreads;
    mine[i] = f < slots ? ids[f] : 0;
  }
  // slots (low half) and entries (high half) of the experts before a thread's
  int c[kOwn], own = 0;
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    const int e = tid * kOwn + i, n = e < a.E ? __popc(mask[e]) : 0;
    c[i] = n | ((n + kEntry - 1) / kEntry) << 16;
    own += c[i];
  }
  int before = own;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, before, d);
    if (lane >= d) before += v;
  }
  if (lane == 31) totals[warp] = before;
  before -= own;
  __syncthreads();
  int all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const int v = totals[w];
    before += w < warp ? v : 0;
    all += v;
  }
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    const int e = tid * kOwn + i, n = c[i] & 0xFFFF, first = before & 0xFFFF;
    for (int j = 0; j * kEntry < n; ++j) {
      r.expert[(before >> 16) + j] = (uint16_t)e;
      r.start[(before >> 16) + j] = (uint16_t)(first + j * kEntry);
    }
    if (n > 0) index[e] = (uint16_t)first;
    before += c[i];
  }
  if (tid == 0) {
    r.n = all >> 16;
    r.start[all >> 16] = (uint16_t)(all & 0xFFFF);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int f = tid + i * kThreads;
    if (f < slots) {
      const int e = mine[i], t = f / a.by_k, at = index[e] + __popc(mask[e] & ((1u << t) - 1));
      r.slot[at] = (uint16_t)f;
      r.token[at] = (uint8_t)t;
    }
  }
  __syncthreads();
}

// A row of activations in shared memory: `parts` f16 numbers to an element, blocks x
// 128 of each; the 16 bytes keep neighbouring rows off each other's banks. After
// the rows, each row's blocks' scales.
__host__ __device__ inline int row_bytes(int parts, int blocks) { return parts * blocks * 256 + 16; }
__host__ __device__ inline int64_t rows_bytes(int64_t rows, int parts, int64_t blocks) {
  return rows * (parts * blocks * 256 + 16 + 4 * blocks);
}
__host__ __device__ inline int most_blocks(int rows, int parts, int bytes) {
  return (bytes / rows - 16) / (parts * 256 + 4);
}

// Units [first, end) whose activations lie in shared memory together: `rows` of
// them from slot[entry] on (all tokens or slots in their order, where all fit),
// `blocks` blocks of K at a time. At most 1024 units: their blocks times the warps
// are counted in 32 bits.
struct Pass {
  int first, end, entry, rows, blocks;
  bool whole;   // K at once
  // a warp's run of the pass's blocks, counted unit by unit, where K is taken at once
  __device__ __forceinline__ int from(int warp) const {
    return (end - first) * blocks * warp / kWarps;
  }
};

// A block's units [u0, u1), and where it has all experts of its columns, its tiles
// of 16 columns.
struct Run {
  int u0, u1, tile0, tile1;
};
template <bool kDown>
__device__ __forceinline__ Run run_of(const FewArgs& a, const Route& r) {
  const uint32_t b = blockIdx.x, n = gridDim.x;
  Run v{};
  if (kDown && a.resident) {
    v.tile0 = (int)((uint32_t)a.tiles * b / n);
    v.tile1 = (int)((uint32_t)a.tiles * (b + 1) / n);
    v.u1 = (v.tile1 - v.tile0 + 1) / 2 * r.n;
  } else {
    const uint32_t units = (uint32_t)r.n * a.upe;   // below 2^27
    const uint32_t q = units / n, more = units - q * n;
    v.u0 = (int)(b * q + min(b, more));
    v.u1 = (int)(v.u0 + q + (b < more ? 1 : 0));
    v.tile1 = a.tiles;
  }
  return v;
}

// A unit's entry and (first) tile. Units are ordered by expert, or by output
// columns (the second kernel with the h of all slots).
template <bool kDown>
__device__ __forceinline__ void decode(const FewArgs& a, const Route& r, const Run& run, int unit, int& x, int& tile) {
  if (kDown && a.resident) {
    const int i = unit / r.n;
    x = unit - i * r.n;
    tile = run.tile0 + 2 * i;
  } else {
    x = unit / a.by_upe;
    tile = (unit - x * a.upe) * (kDown ? 2 : 1);
  }
}

template <int P, bool kDown>
__device__ __forceinline__ Pass pass_at(const FewArgs& a, const Route& r, int u, int u1) {
  Pass p;
  p.first = u;
  p.blocks = a.KB;
  p.whole = true;
  if (a.resident) {
    p.entry = 0;
    p.rows = kDown ? a.T * a.k : a.T;
    p.end = min(u1, u + 1024);
    return p;
  }
  int x = u / a.by_upe;
  p.entry = r.start[x];
  p.rows = r.start[x + 1] - p.entry;
  p.end = min(u1, (x + 1) * a.upe);
  p.whole = rows_bytes(p.rows, P, a.KB) <= kRowsBytes;
  if (p.whole) {
    for (int more = 0; more < 15 && p.end < min(u1, u + 1024); ++more) {
      ++x;
      const int rows = r.start[x + 1] - p.entry;
      if (rows_bytes(rows, P, a.KB) > kRowsBytes) break;
      p.rows = rows;
      p.end = min(u1, (x + 1) * a.upe);
    }
    p.end = min(p.end, u + 1024);
  } else {
    p.end = min(p.end, u + 2 * kWarps);
    p.blocks = most_blocks(p.rows, P, kRowsBytes);
  }
  return p;
}

__device__ __forceinline__ void load_row(Raw16<float>& raw, const float* from) {   // h: written by other SMs
#pragma unroll
  for (int j = 0; j < 4; ++j) raw.w[j] = __ldcg(reinterpret_cast<const uint4*>(from) + j);
}
template <typename T>
__device__ __forceinline__ void load_row(Raw16<T>& raw, const T* from) {
#pragma unroll
  for (int j = 0; j < (int)sizeof(T); ++j) raw.w[j] = reinterpret_cast<const uint4*>(from)[j];
}

// The pass's activations of blocks [b0, b0 + n) into shared memory, by the threads
// from `thread0` on: eight lanes to a block, U blocks of theirs at a time (a load
// from L2 takes one to two microseconds with the codes on their way). Zeros past the
// row's end.
template <typename T, int P, bool kDown>
__device__ __forceinline__ void stage_rows(const FewArgs& a, const Route& r, const Pass& p, int b0, int n, uint8_t* xs,
                                           int thread0 = 0) {
  constexpr int U = 2;
  const int bytes = row_bytes(P, p.blocks), piece = threadIdx.x & 7, step = (32 * kWarps - thread0) / 8;
  float* scale = reinterpret_cast<float*>(xs + p.rows * bytes);
  // a block's row, and how far the threads' next blocks are
  int b = (threadIdx.x - thread0) >> 3;
  int row = n == a.KB ? b / a.by_KB : b / n, rows_on = n == a.KB ? step / a.by_KB : step / n;
  b -= row * n;
  const int on = step - rows_on * n;
  while (__any_sync(0xFFFFFFFFu, row < p.rows)) {
    Raw16<T> raw[U];
    int rows[U], blocks[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int col = (b0 + b) * kBlock + piece * 16;
      rows[j] = row;
      blocks[j] = b;
      raw[j].zero();
      if (row < p.rows && col < a.width) {
        const int at = a.resident ? row : kDown ? r.slot[p.entry + row] : r.token[p.entry + row];
        load_row(raw[j], static_cast<const T*>(a.src) + at * a.lds + col);
      }
      b += on;
      row += rows_on;
      if (b >= n) {
        b -= n;
        ++row;
      }
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      float v[16];
      to_f32(raw[j], v);
      float m = amax16(v);
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
      // 2^e <= m < 2^(e+1), but 2^-100 where less; blocks with an infinity or NaN are not scaled up or down
      int e = (int)((__float_as_uint(m) >> 23) & 255u) - 127;
      e = m < INFINITY ? max(e, -100) : 14;
      const float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
      uint32_t hi[8], lo[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float f0 = v[2 * i] * up, f1 = v[2 * i + 1] * up;
        const __half2 h = __floats2half2_rn(f0, f1);
        hi[i] = *reinterpret_cast<const uint32_t*>(&h);
        if constexpr (P == 2) {
          const float2 t = __half22float2(h);
          const __half2 l =
              __floats2half2_rn(fabsf(t.x) < INFINITY ? f0 - t.x : 0.0f, fabsf(t.y) < INFINITY ? f1 - t.y : 0.0f);
          lo[i] = *reinterpret_cast<const uint32_t*>(&l);
        }
      }
      if (rows[j] < p.rows) {
        // piece 2 q + h lies at 4 h + q, for the lanes that take pieces 2 q + h of the codes
        uint4* out =
            reinterpret_cast<uint4*>(xs + rows[j] * bytes + blocks[j] * 256 + (piece & 1) * 128 + (piece >> 1) * 32);
        out[0] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        out[1] = make_uint4(hi[4], hi[5], hi[6], hi[7]);
        if constexpr (P == 2) {
          uint4* low = out + p.blocks * 16;
          low[0] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          low[1] = make_uint4(lo[4], lo[5], lo[6], lo[7]);
        }
        if (piece == 0) scale[rows[j] * p.blocks + blocks[j]] = __uint_as_float((uint32_t)(127 - 14 + e) << 23);
      }
    }
  }
}

// The unit after that.
template <bool kDown>
__device__ __forceinline__ void advance(const FewArgs& a, const Route& r, int& x, int& tile) {
  if (kDown && a.resident) {
    if (++x == r.n) {
      x = 0;
      tile += 2;
    }
  } else {
    tile += kDown ? 2 : 1;
    if (tile >= (kDown ? a.tiles : a.upe)) {
      tile = 0;
      ++x;
    }
  }
}

// The codes that a warp reads, in order. Where K is taken at once, the warps share
// the pass's blocks evenly, unit by unit: a warp's run may start and end within a
// unit. Otherwise a warp has units of its own, once for each piece of K. Runs
// ahead of the products by the ring's length.
template <int P, bool kDown>
struct Stream {
  Pass p;
  Run run;
  int unit, x, tile, b0;
  int left;                 // blocks of the run after this unit's
  int here;                 // blocks of this unit left, with the next one
  int b, row;               // the next block; the unit's first row among all experts'
  const float* sf;          // lane 0: the scales of its first tile's rows, lane 1: its second's
  bool live, two;           // the unit has a second tile

  __device__ __forceinline__ void at_unit(const FewArgs& a, const Route& r, int first, int n) {
    row = r.expert[x] * (int)a.rows + tile * 16;
    two = !kDown || tile + 1 < run.tile1;
    // (where there is no second tile, the first's scale stands in)
    const int at = (threadIdx.x & 31) == 0 || !two ? tile : kDown ? tile + 1 : tile + a.tiles / 2;
    sf = a.sf + (r.expert[x] * a.row_blocks + at / 8) * a.KB;
    b = first;
    here = n;
  }
  __device__ __forceinline__ void enter(const FewArgs& a, const Route& r, int u, int warp) {
    live = false;
    for (; u < run.u1; u = p.end) {
      p = pass_at<P, kDown>(a, r, u, run.u1);
      if (p.whole) {
        const int f = p.from(warp), n = p.from(warp + 1) - f;
        if (n == 0) continue;
        unit = f / a.by_KB;
        const int first = f - unit * a.KB;
        unit += p.first;
        decode<kDown>(a, r, run, unit, x, tile);
        at_unit(a, r, first, min(n, a.KB - first));
        left = n - here;
      } else {
        unit = u + warp;
        if (unit >= p.end) continue;
        b0 = 0;
        decode<kDown>(a, r, run, unit, x, tile);
        at_unit(a, r, 0, p.blocks);
      }
      live = true;
      return;
    }
  }
  // the unit's blocks are used up
  __device__ __forceinline__ void next_unit(const FewArgs& a, const Route& r, int warp) {
    if (p.whole) {
      if (left == 0) {
        enter(a, r, p.end, warp);
      } else {
        advance<kDown>(a, r, x, tile);
        at_unit(a, r, 0, min(left, a.KB));
        left -= here;
      }
      return;
    }
    unit += kWarps;
    if (unit >= p.end) {
      b0 += p.blocks;
      if (b0 >= a.KB) {
        enter(a, r, p.end, warp);
        return;
      }
      unit = p.first + warp;
    }
    decode<kDown>(a, r, run, unit, x, tile);
    at_unit(a, r, b0, min(p.blocks, a.KB - b0));
  }
};

__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ void from_float(__nv_bfloat16& d, float v) { d = __float2bfloat16_rn(v); }
__device__ __forceinline__ void from_float(__half& d, float v) { d = __float2half_rn(v); }
__device__ __forceinline__ void from_float(float& d, float v) { d = v; }

// y of n columns from c0 on, of all tokens, by one warp.
template <typename Y>
__device__ __forceinline__ void join_experts(const FewArgs& a, const Route& r, int c0, int n) {
  const int lane = threadIdx.x & 31;
  if (lane >= n) return;
  // eight tokens' loads at a time are on their way together
  const int64_t c = c0 + lane;
  for (int t0 = 0; t0 < a.T; t0 += 8) {
    float s[8] = {};
    for (int j = 0; j < a.k; j += 2) {
      float o[2][8];
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (t0 + i / 2 < a.T && j + i % 2 < a.k)
          o[i % 2][i / 2] = __ldcg(a.dst + (int64_t)((t0 + i / 2) * a.k + j + i % 2) * a.ldd + c);
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (t0 + i / 2 < a.T && j + i % 2 < a.k)
          s[i / 2] = fmaf(r.weight[(t0 + i / 2) * a.k + j + i % 2], o[i % 2][i / 2], s[i / 2]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int t = t0 + i;
      if (t >= a.T) break;
      if (a.residual) s[i] += to_float(static_cast<const Y*>(a.residual)[t * a.ldr + c]);
      from_float(static_cast<Y*>(a.y)[t * a.ldy + c], s[i]);
    }
  }
}

// T: type of the source rows; Y: of y. P: f16 numbers to an activation.
template <typename T, typename Y, int P, bool kDown>
__global__ void __launch_bounds__(32 * kWarps, 1)
    few_tokens_kernel(const __grid_constant__ CUtensorMap map, const FewArgs a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
  uint8_t* ring = smem + warp * (kStages * kStageBytes);                                 // 1024-byte aligned stages
  float4* parts = reinterpret_cast<float4*>(smem + kWarps * kStages * kStageBytes);   // sums of parts, two a warp
  Route& r = *reinterpret_cast<Route*>(parts + kWarps * 4 * 32);
  uint64_t* bars = reinterpret_cast<uint64_t*>(&r + 1);
  float* sfs = reinterpret_cast<float*>(bars + kWarps * kStages) + warp * (kStages * 2);       // a stage's scales
  uint8_t* xs = reinterpret_cast<uint8_t*>(bars + kWarps * kStages * 2);
  const uint32_t ring_at = smem_addr(ring), bar_at = smem_addr(bars + warp * kStages);
  volatile int* gave_up = &r.gave_up;
  if (lane == 0) {
    if (warp == 0) {
      prefetch_tensormap(&map);
      *gave_up = 0;
      mbar_init(smem_addr(&r.never), 1);
    }
    for (int i = 0; i < kStages; ++i) mbar_init(bar_at + 8 * i, 3);   // codes, and two scales
    fence_mbar_init();
  }
  if constexpr (!kDown) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int i = blockIdx.x * 32 * kWarps + tid; i <= a.n_counters; i += gridDim.x * 32 * kWarps) a.counters[i] = 0;
  }
  // the warps without a token to route bring the activations meanwhile (x)
  bool staged = !kDown && a.resident && 2 * a.T <= kWarps;
  route_all(a, r, reinterpret_cast<uint32_t*>(smem), [&]() {
    if (staged) stage_rows<T, P, kDown>(a, r, Pass{0, 0, 0, a.T, a.KB, true}, 0, a.KB, xs, 32 * a.T);
  });
  // (the scratch lies where copies go: read and written by the generic proxy before)
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncthreads();
  const Run run = run_of<kDown>(a, r);

  Stream<P, kDown> ahead;
  ahead.run = run;
  ahead.enter(a, r, run.u0, warp);
  const uint64_t policy = l2_policy_evict_first();   // codes are read once
  const uint32_t wait_at = a.test_stall ? smem_addr(&r.never) : bar_at, wait_step = a.test_stall ? 0 : 8;
  uint32_t filled = 0, used = 0, put = 0, get = 0, phase = 0;
  auto fill = [&]() {
    if (ahead.live) {
      const uint32_t stage = ring_at + put * kStageBytes, bar = bar_at + 8 * put;
      if (lane == 0) {
        mbar_arrive_expect_tx(bar, ahead.two ? kStageBytes : kTileBytes);
        tma_load_2d(stage, &map, bar, ahead.b * kBlock, ahead.row, policy);
        if (ahead.two)
          tma_load_2d(stage + kTileBytes, &map, bar, ahead.b * kBlock, ahead.row + (kDown ? 16 : (int)(a.rows / 2)),
                      policy);
      }
      if (lane < 2) {   // the tiles' scales
        cp_async_4(smem_addr(sfs + put * 2 + lane), ahead.sf + ahead.b);
        cp_async_arrive_noinc(bar);
      }
      ++filled;
      ++ahead.b;
      if (--ahead.here == 0) ahead.next_unit(a, r, warp);
    }
    put = put + 1 == kStages ? 0 : put + 1;
  };
  for (int i = 0; i < kStages - 1; ++i) fill();
  // the second kernel's blocks come this far beside the first's
  if constexpr (kDown) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (tid == 0 && __ldcg(a.counters + a.n_counters)) *gave_up = 1;   // h is not complete: no result
  }
  bool ok = true;
  // second kernel, resident: the experts' sums of this block's columns
  float* outs = reinterpret_cast<float*>(xs + rows_bytes(a.T * a.k, P, a.KB));
  const int ncols = (run.tile1 - run.tile0) * 16, col0 = run.tile0 * 16;

  // The sums of blocks [b0, b1) of a unit of entry x, counted from the first in
  // shared memory, added to `sum`.
  auto add_blocks = [&](const Pass& p, int x, int b0, int b1, float (&sum)[2][4]) {
    const int entry = r.start[x], cols = r.start[x + 1] - entry;
    auto row_at = [&](int col) {
      return !a.resident ? entry - p.entry + col : kDown ? (int)r.slot[entry + col] : (int)r.token[entry + col];
    };
    const int bytes = row_bytes(P, p.blocks);
    const float* scales = reinterpret_cast<const float*>(xs + p.rows * bytes);
    // columns past the entry's last read a row that there is; their sums are not used
    const uint8_t* xrow = xs + row_at(min(g, cols - 1)) * bytes + q * 32;
    const float* srow0 = scales + row_at(min(2 * q, cols - 1)) * p.blocks;
    const float* srow1 = scales + row_at(min(2 * q + 1, cols - 1)) * p.blocks;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      __syncwarp();   // the stage before this one is read, and takes the next copies
      if (ok) {
        fill();
        ok = wait_warp(wait_at + wait_step * get, phase, gave_up, a.wait_limit_ns, a.status, kDown ? 52 : 51);
        used += ok;
      }
      const uint8_t* stage = ring + get * kStageBytes;
      const float f0 = sfs[get * 2], f1 = sfs[get * 2 + 1];
      if (++get == kStages) {
        get = 0;
        phase ^= 1;
      }
      float acc[2][P][4];   // MMAs that do not wait for each other: the tiles and the parts apart
      const float zero[4] = {};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t f[2][4][4];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          // rows g and g + 8 of the tile, 16 bytes each, where the copies' swizzle puts them
          const uint8_t* codes = stage + t * kTileBytes + g * 128 + (((2 * q + h) ^ g) << 4);
          const uint4 wl = *reinterpret_cast<const uint4*>(codes), wh = *reinterpret_cast<const uint4*>(codes + 1024);
          const uint32_t lw[4] = {wl.x, wl.y, wl.z, wl.w}, hw[4] = {wh.x, wh.y, wh.z, wh.w};
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            codes_to_f16(lw[s], f[t][s][0], f[t][s][2]);
            codes_to_f16(hw[s], f[t][s][1], f[t][s][3]);
          }
        }
#pragma unroll
        for (int part = 0; part < P; ++part) {
          const uint8_t* at = xrow + part * p.blocks * 256 + b * 256 + h * 128;
          const uint4 x0 = *reinterpret_cast<const uint4*>(at), x1 = *reinterpret_cast<const uint4*>(at + 16);
          float(&d0)[4] = acc[0][part], (&d1)[4] = acc[1][part];
          // (an accumulator's first product needs no zeros in registers)
          if (h == 0) mma_f16(d0, f[0][0], x0.x, x0.y, zero);
          else mma_f16(d0, f[0][0], x0.x, x0.y, d0);
          if (h == 0) mma_f16(d1, f[1][0], x0.x, x0.y, zero);
          else mma_f16(d1, f[1][0], x0.x, x0.y, d1);
          mma_f16(d0, f[0][1], x0.z, x0.w, d0);
          mma_f16(d1, f[1][1], x0.z, x0.w, d1);
          mma_f16(d0, f[0][2], x1.x, x1.y, d0);
          mma_f16(d1, f[1][2], x1.x, x1.y, d1);
          mma_f16(d0, f[0][3], x1.z, x1.w, d0);
          mma_f16(d1, f[1][3], x1.z, x1.w, d1);
        }
      }
      const float x0 = srow0[b], x1 = srow1[b];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const float ft = t ? f1 : f0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float v = acc[t][0][i];
          if constexpr (P == 2) v += acc[t][1][i];
          sum[t][i] = fmaf(v, ft * (i & 1 ? x1 : x0), sum[t][i]);
        }
      }
    }
  };
  // What a unit's sums become.
  auto finish = [&](int x, int tile, const float (&sum)[2][4]) {
    // (parts may be of a warp that gave up; others set the word at any time, so that lanes
    // may read it differently, and what follows takes the whole warp)
    if (__any_sync(0xFFFFFFFFu, !ok || *gave_up)) return;
    const int entry = r.start[x], cols = r.start[x + 1] - entry;
    const bool two = tile + 1 < run.tile1;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int col = 2 * q + i;
      if (col < cols) {
        const int slot = r.slot[entry + col];
        if constexpr (!kDown) {
          float* h = a.dst + slot * a.ldd + tile * 16 + g;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float gate = sum[0][2 * j + i];
            h[8 * j] = gate / (1.0f + expf(-gate)) * sum[1][2 * j + i];
          }
        } else {
          float* out = (a.resident ? outs + slot * ncols - col0 : a.dst + slot * a.ldd) + tile * 16 + g;
          out[0] = sum[0][i];
          out[8] = sum[0][2 + i];
          if (two) {
            out[16] = sum[1][i];
            out[24] = sum[1][2 + i];
          }
        }
      }
    }
    if (kDown && !a.resident) {
      __threadfence();
      __syncwarp();
      int done = 0;
      if (lane == 0) done = atomicAdd(a.counters + tile / 2, 1);
      done = __shfl_sync(0xFFFFFFFFu, done, 0);
      if (done == r.n - 1) {
        __threadfence();
        join_experts<Y>(a, r, tile * 16, two ? 32 : 16);
      }
    }
  };
  auto set = [](float (&to)[2][4], const float (&from)[2][4]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) to[i / 4][i % 4] = from[i / 4][i % 4];
  };
  const float none[2][4] = {};

  for (int u = run.u0; u < run.u1;) {
    const Pass p = pass_at<P, kDown>(a, r, u, run.u1);
    __syncthreads();   // the activations and parts before are used up
    if (!staged) stage_rows<T, P, kDown>(a, r, p, 0, min(p.blocks, a.KB), xs);
    staged = a.resident;
    __syncthreads();
    if (p.whole) {
      const int f0 = p.from(warp), f1 = p.from(warp + 1);
      int open = -1, open_x = 0, open_tile = 0;   // the unit that this warp begins and others end
      int unit = f0 / a.by_KB, b0 = f0 - unit * a.KB, x, tile;
      unit += p.first;
      decode<kDown>(a, r, run, unit, x, tile);
      for (int f = f0; f < f1; ++unit) {
        const int b1 = min(a.KB, b0 + f1 - f);
        float sum[2][4];
        set(sum, none);
        add_blocks(p, x, b0, b1, sum);
        if (b1 - b0 == a.KB) {
          finish(x, tile, sum);
        } else {
          if (b0 == 0) open = unit, open_x = x, open_tile = tile;
#pragma unroll
          for (int t = 0; t < 2; ++t)
            parts[((warp * 2 + (b0 == 0)) * 2 + t) * 32 + lane] =
                make_float4(sum[t][0], sum[t][1], sum[t][2], sum[t][3]);
        }
        f += b1 - b0;
        b0 = 0;
        advance<kDown>(a, r, x, tile);
      }
      __syncthreads();
      if (open >= 0) {
        float sum[2][4];
        const int end = (open - p.first + 1) * a.KB;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          float4 v = parts[((warp * 2 + 1) * 2 + t) * 32 + lane];
          for (int w = warp + 1; w < kWarps && p.from(w) < end; ++w) {
            if (p.from(w) == p.from(w + 1)) continue;   // it has none
            const float4 more = parts[(w * 4 + t) * 32 + lane];
            v.x += more.x, v.y += more.y, v.z += more.z, v.w += more.w;
          }
          sum[t][0] = v.x, sum[t][1] = v.y, sum[t][2] = v.z, sum[t][3] = v.w;
        }
        finish(open_x, open_tile, sum);
      }
    } else {
      float held[2][2][4];   // sums of the warp's two units
      set(held[0], none);
      set(held[1], none);
      for (int k0 = 0; k0 < a.KB; k0 += p.blocks) {
        const int n = min(p.blocks, a.KB - k0);
        if (k0 > 0) {
          __syncthreads();
          stage_rows<T, P, kDown>(a, r, p, k0, n, xs);
          __syncthreads();
        }
        for (int i = 0; i < 2; ++i) {
          const int unit = p.first + warp + i * kWarps;
          if (unit >= p.end) break;
          float sum[2][4];
          if (i) set(sum, held[1]);
          else set(sum, held[0]);
          int x, tile;
          decode<kDown>(a, r, run, unit, x, tile);
          add_blocks(p, x, 0, n, sum);
          if (i) set(held[1], sum);
          else set(held[0], sum);
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int unit = p.first + warp + i * kWarps;
        int x, tile;
        decode<kDown>(a, r, run, unit, x, tile);
        if (unit < p.end) finish(x, tile, held[i]);
      }
    }
    u = p.end;
  }
  if constexpr (kDown) {
    __syncthreads();
    if (a.resident && !*gave_up) {
      for (int i = tid; i < a.T * ncols; i += 32 * kWarps) {
        const int t = i / ncols, c = i - t * ncols;
        float s = 0.0f;
#pragma unroll 4
        for (int j = 0; j < a.k; ++j) s = fmaf(r.weight[t * a.k + j], outs[(t * a.k + j) * ncols + c], s);
        if (a.residual) s += to_float(static_cast<const Y*>(a.residual)[t * a.ldr + col0 + c]);
        from_float(static_cast<Y*>(a.y)[t * a.ldy + col0 + c], s);
      }
    }
  }
  // a warp that gave up tells the second kernel, and waits for its copies in flight
  if (!kDown && !ok && lane == 0) a.counters[a.n_counters] = 1;
  if (!ok && lane == 0)
    for (; used < filled; ++used) drain_wait(bar_at + 8 * (used % kStages), used / kStages & 1u);
}

bool few_shape_ok(int type, int64_t T, int64_t K, int64_t I, int E, int k) {
  return type_ok(type) && T >= 0 && T <= kMaxTokens && K > 0 && K % 16 == 0 && K < (1ll << 20) && I > 0 &&
         I % 16 == 0 && I < (1ll << 20) && E * K < (1ll << 31) && E * 2 * I < (1ll << 31) && k >= 1 && k <= 16 &&
         E >= k && E <= 1024;
}

int64_t up256(int64_t v) { return ceil_div(v, 256) * 256; }

// The workspace: the counters, h and out.
struct FewLayout {
  int64_t h, out, total;
  FewLayout(int64_t T, int64_t K, int64_t I, int k) {
    h = up256((ceil_div(K, 32) + 1) * 4);
    out = h + up256(T * k * I * 4);
    total = out + up256(T * k * K * 4);
  }
};

template <typename T, typename Y, int P, bool kDown>
int launch_few(const CUtensorMap& map, FewArgs& a, int sms, cudaStream_t s) {
  auto kernel = few_tokens_kernel<T, Y, P, kDown>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes) != cudaSuccess) {
    cudaGetLastError();
    return NVFP4MOE_ERR_LAUNCH;
  }
  const int64_t slots = a.T * a.k, most = (slots < a.E ? slots : a.E) * a.upe;
  a.resident = kDown ? rows_bytes(slots, P, a.KB) + slots * ceil_div(a.tiles, sms) * 64 <= kRowsBytes
                     : rows_bytes(a.T, P, a.KB) <= kRowsBytes;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)(kDown && a.resident ? (a.tiles < sms ? a.tiles : sms) : most < sms ? most : sms), 1, 1);
  cfg.blockDim = dim3(32 * kWarps, 1, 1);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = kDown ? 1 : 0;
  cudaLaunchKernelEx(&cfg, kernel, map, (const FewArgs&)a);
  return launch_status();
}

struct FewCall {
  CUtensorMap w1, w2;
  FewArgs up{}, down{};
  int sms;
  cudaStream_t s;
};

// P: f16 numbers to an element of x; h takes two whatever y's type.
template <typename T, int P>
int run_few(FewCall& c) {
  NVFP4_TRY((launch_few<T, T, P, false>(c.w1, c.up, c.sms, c.s)));
  return launch_few<float, T, 2, true>(c.w2, c.down, c.sms, c.s);
}

}  // namespace
}  // namespace nvfp4moe

using namespace nvfp4moe;

extern "C" size_t fp8_moe_few_tokens_workspace_size(int64_t T, int64_t K, int64_t I, int E, int k) {
  if (!few_shape_ok(NVFP4MOE_BF16, T, K, I, E, k)) return 0;
  return (size_t)FewLayout(T, K, I, k).total;
}

extern "C" int fp8_moe_few_tokens(const void* x, int type, int64_t T, int64_t K, int64_t ldx,
                                  const float* router_logits, int64_t I, int E, int k, const uint8_t* w1_codes,
                                  const float* w1_sf, const uint8_t* w2_codes, const float* w2_sf,
                                  const void* residual, int64_t ldr, void* y, int64_t ldy, void* ws, size_t ws_bytes,
                                  void* stream) {
  NVFP4_CHECK(few_shape_ok(type, T, K, I, E, k), NVFP4MOE_ERR_UNSUPPORTED);
  if (T == 0) return NVFP4MOE_OK;
  const int64_t es = type_bytes(type);
  NVFP4_CHECK(x && router_logits && w1_codes && w1_sf && w2_codes && w2_sf && y, NVFP4MOE_ERR_INVALID);
  NVFP4_CHECK(ldx >= K && ldx * es % 16 == 0 && aligned(x, 16) && aligned(router_logits, 4) && aligned(w1_codes, 16) &&
                  aligned(w2_codes, 16) && aligned(w1_sf, 4) && aligned(w2_sf, 4) && ldy >= K && aligned(y, es) &&
                  (!residual || (ldr >= K && aligned(residual, es))),
              NVFP4MOE_ERR_INVALID);
  NVFP4_CHECK(ws && ws_bytes >= fp8_moe_few_tokens_workspace_size(T, K, I, E, k) && aligned(ws, 256),
              NVFP4MOE_ERR_WORKSPACE);
  const int sms = device_num_sms();
  NVFP4_CHECK(sms > 0, NVFP4MOE_ERR_LAUNCH);
  uint8_t* w = static_cast<uint8_t*>(ws);
  const FewLayout L(T, K, I, k);
  FewCall c{};
  c.sms = sms;
  c.s = as_stream(stream);
  NVFP4_CHECK(make_codes_map(&c.w1, w1_codes, E * 2 * I, K, K, 16) && make_codes_map(&c.w2, w2_codes, E * K, I, I, 16),
              NVFP4MOE_ERR_INVALID);
  FewArgs &up = c.up, &down = c.down;
  up.logits = router_logits, up.T = (int)T, up.E = E, up.k = k, up.by_k = Divisor(k);
  up.counters = reinterpret_cast<int*>(w), up.n_counters = (int)ceil_div(K, 32);
  up.wait_limit_ns = wait_limit_ns(), up.status = device_status_word(), up.test_stall = test_stall_on();
  NVFP4_CHECK(up.status, NVFP4MOE_ERR_LAUNCH);
  down = up;
  auto half = [](FewArgs& a, const void* src, int64_t lds, int64_t width, const float* sf, int64_t rows, uint8_t* dst,
                 int64_t ldd) {
    a.src = src, a.lds = lds, a.width = (int)width, a.KB = (int)ceil_div(width, kBlock), a.sf = sf;
    a.rows = rows, a.row_blocks = ceil_div(rows, kBlock), a.tiles = (int)(rows / 16), a.upe = (a.tiles + 1) / 2;
    a.dst = reinterpret_cast<float*>(dst), a.ldd = ldd;
    a.by_upe = Divisor(a.upe), a.by_KB = Divisor(a.KB);
  };
  half(up, x, ldx, K, w1_sf, 2 * I, w + L.h, I);
  half(down, w + L.h, I, I, w2_sf, K, w + L.out, K);
  down.y = y, down.ldy = ldy, down.residual = residual, down.ldr = ldr;
  if (type == NVFP4MOE_BF16) return run_few<__nv_bfloat16, 1>(c);
  if (type == NVFP4MOE_F16) return run_few<__half, 1>(c);
  return run_few<float, 2>(c);
}
