// Tokens in expert order and back, with routing weights, and the gradients.
//
// With p(t, j) = flat_to_perm[t * k + j], the row of slot j of token t:
//   sort             rows[p(t,j)] = w[t,j] * x[t]
//   sort backward    dx[t] = sum_j w[t,j] * d_rows[p(t,j)],  d_w[t,j] = <x[t], d_rows[p(t,j)]>
//   unsort           y[t]  = sum_j w[t,j] * rows[p(t,j)]
//   unsort backward  d_rows[p(t,j)] = w[t,j] * dy[t],        d_w[t,j] = <dy[t], rows[p(t,j)]>
// Two kernels do all four: one spreads a token row over its k rows, the other
// sums the k rows of a token; each takes the dot products of d_w along, from
// data that it reads anyway (the sum) or that the spread reads beside it.
// Everything is read once and written once, so HBM bounds them.
#include "common.cuh"

#include <cuda_fp16.h>

namespace nvfp4moe {
namespace {

constexpr int kMaxK = 16;

struct Args {
  const void* token_in;    // spread: the token rows; collect with dots: the token rows of the dots
  void* token_out;         // collect: the sums
  int64_t ldt_in, ldt_out;
  const void* rows_in;     // collect: the rows; spread with dots: the rows of the dots
  void* rows_out;          // spread: the rows written
  int64_t ldr_in, ldr_out;
  int64_t n_rows;          // rows that flat_to_perm may name
  const int32_t* f2p;
  const float* w;          // (T, k) or null: all ones
  float* d_w;              // (T, k), with dots
  int64_t T, K;
  int k;
  int* status;
};

template <typename T> struct Elem;
template <> struct Elem<__nv_bfloat16> {
  static __device__ __forceinline__ float get(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
};
template <> struct Elem<__half> {
  static __device__ __forceinline__ float get(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half put(float v) { return __float2half_rn(v); }
};
template <> struct Elem<float> {
  static __device__ __forceinline__ float get(float v) { return v; }
  static __device__ __forceinline__ float put(float v) { return v; }
};

// V consecutive elements: 16 bytes where all rows start on 16-byte boundaries,
// else two elements, of which rows of an odd width hold every other one's pairs
// unaligned (the same for all lanes of a warp).
template <typename T, int V>
struct alignas(V * sizeof(T)) Pack {
  T e[V];
};

// What is read for a pack: nothing but loads, so that those of all of a token's
// rows are in flight before the first is used. A pair of 16-bit elements comes
// from the two 4-byte words at and after it (one element before the pair to two
// behind it: columns [kHead, K - kTail) are read in pairs, the others one by
// one), a pair of f32 from two loads.
template <int V> constexpr int kHead = V > 2 ? 0 : 2;
template <int V> constexpr int kTail = V > 2 ? 0 : 2;

template <typename T, int V>
struct Raw {
  Pack<T, V> v;
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (V > 2) {
      v = *reinterpret_cast<const Pack<T, V>*>(p);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) v.e[i] = p[i];
    }
  }
  __device__ __forceinline__ Pack<T, V> get(const T*) const { return v; }
};

template <typename T>
struct Words {
  uint32_t w0, w1;
  __device__ __forceinline__ void load(const T* p) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(reinterpret_cast<uintptr_t>(p) & ~static_cast<uintptr_t>(3));
    w0 = w[0];
    w1 = w[1];
  }
  __device__ __forceinline__ Pack<T, 2> get(const T* p) const {
    const uint32_t both = __funnelshift_r(w0, w1, static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 2) * 8);
    return *reinterpret_cast<const Pack<T, 2>*>(&both);
  }
};
template <> struct Raw<__nv_bfloat16, 2> : Words<__nv_bfloat16> {};
template <> struct Raw<__half, 2> : Words<__half> {};

template <typename T, int V>
__device__ __forceinline__ void store_pack(T* p, const Pack<T, V>& v) {
  using P = Pack<T, V>;
  if (V > 2 || reinterpret_cast<uintptr_t>(p) % sizeof(P) == 0) {
    *reinterpret_cast<P*>(p) = v;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = v.e[i];
  }
}

// A block deals with one token, or with four, a warp each.
template <int TOKENS>
__device__ __forceinline__ void sync_token() {
  if constexpr (TOKENS > 1) __syncwarp();
  else __syncthreads();
}

// The rows of a token's k slots (-1 for a slot without one) and its weights.
// A row outside [0, n_rows) is an error of the caller's: recorded, and taken
// as no row. A negative entry is a dropped slot.
template <int TOKENS>
__device__ __forceinline__ void load_slots(const Args& a, int64_t t, int64_t* row, float* wt) {
  if ((int)threadIdx.x < a.k) {
    int64_t r = a.f2p[t * a.k + threadIdx.x];
    if (r >= a.n_rows) {
      if (atomicCAS(&a.status[0], 0, NVFP4MOE_ERR_INVALID) == 0) a.status[1] = 20;
      r = -1;
    }
    row[threadIdx.x] = r;
    wt[threadIdx.x] = a.w ? a.w[t * a.k + threadIdx.x] : 1.0f;
  }
  sync_token<TOKENS>();
}

// The slots of a block's tokens, in shared memory.
template <int TOKENS>
struct Slots {
  int64_t row[TOKENS][kMaxK];
  float wt[TOKENS][kMaxK];
};

// A token's, as its threads read them: kHeld, from registers, else from shared
// memory as they are needed.
template <int TOKENS, int KM, bool kHeld>
struct TokenSlots {
  const Slots<TOKENS>& s;
  int k, held_row[KM];
  float held_wt[KM];
  __device__ __forceinline__ TokenSlots(const Slots<TOKENS>& slots, int n) : s(slots), k(n) {
    if constexpr (kHeld) {
#pragma unroll
      for (int j = 0; j < KM; ++j) {
        held_row[j] = j < k ? (int)s.row[threadIdx.y][j] : -1;
        held_wt[j] = j < k ? s.wt[threadIdx.y][j] : 0.0f;
      }
    }
  }
  __device__ __forceinline__ bool has(int j) const {
    if constexpr (kHeld) return held_row[j] >= 0;
    else return j < k && s.row[0][j] >= 0;
  }
  __device__ __forceinline__ int64_t row(int j) const {
    if constexpr (kHeld) return held_row[j];
    else return s.row[0][j];
  }
  __device__ __forceinline__ float wt(int j) const {
    if constexpr (kHeld) return held_wt[j];
    else return s.wt[0][j];
  }
};

// Sums of KM values over the block in a fixed order; thread j < k writes slot j.
template <int NT, int TOKENS, int KM>
__device__ __forceinline__ void store_dots(const Args& a, int64_t t, const float (&dot)[KM], const int64_t* row) {
  __shared__ float parts[TOKENS][NT / 32][KM];
  float(&part)[NT / 32][KM] = parts[TOKENS > 1 ? threadIdx.y : 0];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int j = 0; j < KM; ++j) {
    float v = dot[j];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (lane == 0) part[warp][j] = v;
  }
  sync_token<TOKENS>();
  if ((int)threadIdx.x < a.k) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) s += part[i][threadIdx.x];
    a.d_w[t * a.k + threadIdx.x] = row[threadIdx.x] >= 0 ? s : 0.0f;
  }
}

// Slots held in registers help where they leave enough of them: the spread with
// dots of 16-byte pieces of 16-bit elements for more than four slots (2048 x 4096,
// k = 8, with the sum before it 80.5 us against 84.5, 256 x 7168 13.8 against 16.8).
// The sums and pairs of elements lose by it (8192 x 401 63 us against 41), f32 and
// four slots gain nothing.
template <int V, int KM, int TOKENS, bool kSpread, bool kDot>
constexpr bool kHeld = TOKENS > 1 || (V == 8 && KM > 4 && kSpread && kDot);

// One token's row to its k rows. KM >= k slots are unrolled.
template <typename T, int V, int KM, int NT, int TOKENS, bool kDot>
__global__ void __launch_bounds__(NT * TOKENS) spread_kernel(const Args a) {
  __shared__ Slots<TOKENS> slots;
  const int local = TOKENS > 1 ? threadIdx.y : 0;
  const int64_t t = (int64_t)blockIdx.x * TOKENS + local;
  if (TOKENS > 1 && t >= a.T) return;
  load_slots<TOKENS>(a, t, slots.row[local], slots.wt[local]);
  const TokenSlots<TOKENS, KM, kHeld<V, KM, TOKENS, true, kDot>> slot(slots, a.k);
  const T* src = static_cast<const T*>(a.token_in) + t * a.ldt_in;
  float dot[KM];
#pragma unroll
  for (int j = 0; j < KM; ++j) dot[j] = 0.0f;
  const int64_t head = kHead<V>, whole = a.K >= head + kTail<V> + V ? head + (a.K - head - kTail<V>) / V * V : 0;
  // the block's share of the columns (all of them with dots)
  const int part = kDot ? 0 : blockIdx.y, parts = kDot ? 1 : gridDim.y;
  for (int64_t c = head + (part * NT + threadIdx.x) * V; c < whole; c += parts * NT * V) {
    using P = Pack<T, V>;
    Raw<T, V> xr, o[KM];
    xr.load(src + c);
    if constexpr (kDot) {
#pragma unroll
      for (int j = 0; j < KM; ++j)
        if (slot.has(j))
          o[j].load(static_cast<const T*>(a.rows_in) + slot.row(j) * a.ldr_in + c);
    }
    const P x = xr.get(src + c);
#pragma unroll
    for (int j = 0; j < KM; ++j) {
      if (slot.has(j)) {
        P y, d;
        if constexpr (kDot) d = o[j].get(static_cast<const T*>(a.rows_in) + slot.row(j) * a.ldr_in + c);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float v = Elem<T>::get(x.e[i]);
          y.e[i] = Elem<T>::put(slot.wt(j) * v);
          if constexpr (kDot) dot[j] = fmaf(v, Elem<T>::get(d.e[i]), dot[j]);
        }
        store_pack<T, V>(static_cast<T*>(a.rows_out) + slot.row(j) * a.ldr_out + c, y);
      }
    }
  }
  for (int64_t i = part * NT + threadIdx.x; i < a.K - (whole > 0 ? whole - head : 0); i += parts * NT) {   // the other columns
    const int64_t c = whole > 0 && i >= head ? whole + i - head : i;
    const float v = Elem<T>::get(src[c]);
#pragma unroll
    for (int j = 0; j < KM; ++j) {
      if (slot.has(j)) {
        static_cast<T*>(a.rows_out)[slot.row(j) * a.ldr_out + c] = Elem<T>::put(slot.wt(j) * v);
        if constexpr (kDot)
          dot[j] = fmaf(v, Elem<T>::get(static_cast<const T*>(a.rows_in)[slot.row(j) * a.ldr_in + c]), dot[j]);
      }
    }
  }
  if constexpr (kDot) store_dots<NT, TOKENS, KM>(a, t, dot, slots.row[local]);
}

// The weighted sum of a token's k rows, in j order, rounded once.
template <typename T, int V, int KM, int NT, int TOKENS, bool kDot>
__global__ void __launch_bounds__(NT * TOKENS) collect_kernel(const Args a) {
  __shared__ Slots<TOKENS> slots;
  const int local = TOKENS > 1 ? threadIdx.y : 0;
  const int64_t t = (int64_t)blockIdx.x * TOKENS + local;
  if (TOKENS > 1 && t >= a.T) return;
  load_slots<TOKENS>(a, t, slots.row[local], slots.wt[local]);
  const TokenSlots<TOKENS, KM, kHeld<V, KM, TOKENS, false, kDot>> slot(slots, a.k);
  const T* rows = static_cast<const T*>(a.rows_in);
  const T* tok = kDot ? static_cast<const T*>(a.token_in) + t * a.ldt_in : nullptr;
  T* out = static_cast<T*>(a.token_out) + t * a.ldt_out;
  float dot[KM];
#pragma unroll
  for (int j = 0; j < KM; ++j) dot[j] = 0.0f;
  const int64_t head = kHead<V>, whole = a.K >= head + kTail<V> + V ? head + (a.K - head - kTail<V>) / V * V : 0;
  // the block's share of the columns (all of them with dots)
  const int part = kDot ? 0 : blockIdx.y, parts = kDot ? 1 : gridDim.y;
  for (int64_t c = head + (part * NT + threadIdx.x) * V; c < whole; c += parts * NT * V) {
    using P = Pack<T, V>;
    Raw<T, V> r[KM], xr;
#pragma unroll
    for (int j = 0; j < KM; ++j)
      if (slot.has(j)) r[j].load(rows + slot.row(j) * a.ldr_in + c);
    P x;
    if constexpr (kDot) {
      xr.load(tok + c);
      x = xr.get(tok + c);
    }
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.0f;
#pragma unroll
    for (int j = 0; j < KM; ++j) {
      if (slot.has(j)) {
        const P d = r[j].get(rows + slot.row(j) * a.ldr_in + c);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float v = Elem<T>::get(d.e[i]);
          acc[i] = fmaf(slot.wt(j), v, acc[i]);
          if constexpr (kDot) dot[j] = fmaf(Elem<T>::get(x.e[i]), v, dot[j]);
        }
      }
    }
    P y;
#pragma unroll
    for (int i = 0; i < V; ++i) y.e[i] = Elem<T>::put(acc[i]);
    store_pack<T, V>(out + c, y);
  }
  for (int64_t i = part * NT + threadIdx.x; i < a.K - (whole > 0 ? whole - head : 0); i += parts * NT) {
    const int64_t c = whole > 0 && i >= head ? whole + i - head : i;
    float acc = 0.0f;
    const float x = kDot ? Elem<T>::get(tok[c]) : 0.0f;
#pragma unroll
    for (int j = 0; j < KM; ++j) {
      if (slot.has(j)) {
        const float v = Elem<T>::get(rows[slot.row(j) * a.ldr_in + c]);
        acc = fmaf(slot.wt(j), v, acc);
        if constexpr (kDot) dot[j] = fmaf(x, v, dot[j]);
      }
    }
    out[c] = Elem<T>::put(acc);
  }
  if constexpr (kDot) store_dots<NT, TOKENS, KM>(a, t, dot, slots.row[local]);
}

template <typename T, int V, int KM, int NT, bool kSpread, bool kDot, int TOKENS = 1>
void launch_nt(const Args& a, int parts, cudaStream_t s) {
  const dim3 grid((unsigned)ceil_div(a.T, TOKENS), (unsigned)parts), block(NT, TOKENS);
  if constexpr (kSpread) spread_kernel<T, V, KM, NT, TOKENS, kDot><<<grid, block, 0, s>>>(a);
  else collect_kernel<T, V, KM, NT, TOKENS, kDot><<<grid, block, 0, s>>>(a);
}

// Blocks of 64 threads for the sums and the dot products (128 for pairs of
// 16-bit elements, which take more rounds): more blocks in different phases to
// an SM (loads, stores, reduction). 8192 x 7168 BF16, k = 8: sum 163 us against
// 187 with 256 threads, spread with dots 322 against 477 (300 since its slots are
// in registers), sum with dots 184 against 215; pairs, 4096 x 7166: spread with dots 242 against 269 with 64. The
// plain spread is better with 256 (162 against 176). Short rows leave threads of
// such blocks idle, so they get a warp (forward and backward of weighted rows, 8192
// tokens, k = 8, with a warp / 64, or 128 for pairs: 64 columns 18.2 / 26.0 us, 401
// 56.6 / 63.7, 1024 84.1 / 88.1), and the middle of the range 64 threads in the plain
// spread; spread and sum of 8192 BF16 tokens, k = 8, with a warp / 64 (the sum
// of pairs 128) / 256 threads for the spread: 64 columns 12.6 / 14.6 / 26.0 us,
// 401 (201 pairs) 40.5 / 44.7 / 46.6, 500 (250 pairs) 49.4 / 47.9 / 51.4, 2048 (256
// pieces of 16 bytes) 106.0 / 104.5 / 105.1. With few tokens the columns of a
// token are divided over blocks, or, where a block has to see all of them for
// its dot products, its 256 threads (512 for many pairs: 32 x 7167 BF16 9.5 us
// against 11.2) see them in fewer rounds (128 tokens: 6.1 against 11.9; from four
// tokens an SM on, 608: 38.6 against 31.9).
// Many tokens of a round or two of a warp go four to a block, a warp each, since
// the blocks' starts are what takes the time: 30000 x 64, k = 2, 17.9 us against
// 34.0, 8192 x 64, k = 8, 11.8 against 12.5; but 384 columns, k = 8, 26.9 against
// 26.1. Fewer tokens than 16 an SM are started in time one by one.
// The bounds are in packs, and F32's packs of four elements behave as the 16-bit
// types' of eight. F32, the four weighted calls (spread, sum, spread and sum with
// dots), this rule / the other side of it:
//   four tokens to a block / one:  30000 x 64, k = 2, 9.2, 9.8, 12.3, 11.3 / 17.3,
//     17.3, 17.5, 17.3; 8192 x 128, k = 8, 7.5, 5.9, 11.1, 7.5 / 6.7, 6.2, 10.3,
//     7.5; the far corner of the rule, 30000 x 128, k = 8, 26.5, 33.9, 50.7, 38.1 /
//     26.6, 26.7, 49.2, 32.3 (BF16, 256 columns: 28.1, 36.7, 61.5, 42.6 / 27.4,
//     34.6, 58.8, 40.5)
//   a warp / 64 threads, k = 8:  8192 x 800 46.1, 40.8, 73.8, 45.0 / 43.6, 41.3,
//     75.3, 48.1; 2000 x 600 7.3, 6.0, 9.4, 5.7 / 7.8, 6.0, 10.6, 7.2
//   64 / 256 threads for the plain spread:  8192 x 1200, k = 8, 63.0 / 68.5; x 1600
//     81.5 / 78.4; k = 2, 23.1 / 30.6 and 30.5 / 34.4
//   with dots, 512 threads for many pairs / 256, k = 8:  32 x 7167 9.5, 6.4 / 10.5,
//     7.0; 150 x 10001 16.8, 8.2 / 24.6, 9.0 (BF16 13.9, 10.8 / 19.1, 15.5)
//   with dots, 256 threads for few tokens / as for many, k = 8:  300 x 7168 22.1,
//     8.5 / 36.7, 20.3; 600 x 4096 28.8, 12.4 / 31.5, 17.1; 600 x 256, the far
//     corner, 4.6, 4.4 / 3.7, 3.2
template <typename T, int V, int KM>
void launch_v(const Args& a, bool spread, bool dot, cudaStream_t s) {
  constexpr int NT = V == 2 && sizeof(T) == 2 ? 128 : 64;
  const int64_t sms = device_num_sms();
  const int64_t packs = ceil_div(a.K, V);
  auto parts = [&](int threads, int64_t blocks) {
    const int64_t most = ceil_div(packs, threads), want = ceil_div(blocks, a.T);
    return (int)(most < want ? (most > 0 ? most : 1) : want);
  };
  if (packs <= (KM <= 4 ? 64 : 32) && a.T >= 16 * sms) {
    if (spread && dot) launch_nt<T, V, KM, 32, true, true, 4>(a, 1, s);
    else if (spread) launch_nt<T, V, KM, 32, true, false, 4>(a, 1, s);
    else if (dot) launch_nt<T, V, KM, 32, false, true, 4>(a, 1, s);
    else launch_nt<T, V, KM, 32, false, false, 4>(a, 1, s);
  } else if (!dot) {
    if (packs <= 224) {
      if (spread) launch_nt<T, V, KM, 32, true, false>(a, parts(32, 16 * sms), s);
      else launch_nt<T, V, KM, 32, false, false>(a, parts(32, 16 * sms), s);
    } else if (!spread) {
      launch_nt<T, V, KM, NT, false, false>(a, parts(NT, 16 * sms), s);
    } else if (packs < 512) {
      launch_nt<T, V, KM, 64, true, false>(a, parts(64, 16 * sms), s);
    } else {
      launch_nt<T, V, KM, 256, true, false>(a, parts(256, 4 * sms), s);
    }
  } else if (V == 2 && KM <= 8 && a.T < sms && packs >= 2048) {
    if constexpr (V == 2 && KM <= 8) {
      if (spread) launch_nt<T, V, KM, 512, true, true>(a, 1, s);
      else launch_nt<T, V, KM, 512, false, true>(a, 1, s);
    }
  } else if (a.T < 4 * sms) {
    if (spread) launch_nt<T, V, KM, 256, true, true>(a, 1, s);
    else launch_nt<T, V, KM, 256, false, true>(a, 1, s);
  } else if (packs <= 224) {
    if (spread) launch_nt<T, V, KM, 32, true, true>(a, 1, s);
    else launch_nt<T, V, KM, 32, false, true>(a, 1, s);
  } else {
    if (spread) launch_nt<T, V, KM, NT, true, true>(a, 1, s);
    else launch_nt<T, V, KM, NT, false, true>(a, 1, s);
  }
}

// 16-byte accesses where every row of every operand starts on a 16-byte
// boundary, pairs of elements otherwise (4096 x 7167 BF16, k = 8, sum: 131 us
// against 166 with single elements; 4096 x 7168: 88).
template <typename T>
void launch_t(const Args& a, bool spread, bool dot, cudaStream_t s) {
  constexpr int V = 16 / (int)sizeof(T);
  auto whole = [](const void* p, int64_t ld) { return !p || (aligned(p, 16) && ld * (int64_t)sizeof(T) % 16 == 0); };
  const bool wide = whole(a.token_in, a.ldt_in) && whole(a.token_out, a.ldt_out) && whole(a.rows_in, a.ldr_in) &&
                    whole(a.rows_out, a.ldr_out);
  if (wide) {
    if (a.k <= 4) launch_v<T, V, 4>(a, spread, dot, s);
    else if (a.k <= 8) launch_v<T, V, 8>(a, spread, dot, s);
    else launch_v<T, V, 16>(a, spread, dot, s);
  } else {
    if (a.k <= 4) launch_v<T, 2, 4>(a, spread, dot, s);
    else if (a.k <= 8) launch_v<T, 2, 8>(a, spread, dot, s);
    else launch_v<T, 2, 16>(a, spread, dot, s);
  }
}

int launch(Args& a, int type, bool spread, bool dot, void* stream) {
  a.status = device_status_word();
  NVFP4_CHECK(a.status, NVFP4MOE_ERR_LAUNCH);
  cudaStream_t s = as_stream(stream);
  if (type == NVFP4MOE_BF16) launch_t<__nv_bfloat16>(a, spread, dot, s);
  else if (type == NVFP4MOE_F16) launch_t<__half>(a, spread, dot, s);
  else launch_t<float>(a, spread, dot, s);
  return launch_status();
}

int check_sizes(int type, int64_t T, int64_t K, int k, int64_t n_rows) {
  NVFP4_CHECK(type == NVFP4MOE_BF16 || type == NVFP4MOE_F16 || type == NVFP4MOE_F32, NVFP4MOE_ERR_UNSUPPORTED);
  NVFP4_CHECK(T >= 0 && K >= 0 && K < (1ll << 30) && k >= 1 && k <= kMaxK && n_rows >= 0 && T < (1ll << 31) &&
                  T * k < (1ll << 31),
              NVFP4MOE_ERR_UNSUPPORTED);
  return NVFP4MOE_OK;
}

bool element_aligned(const void* p, int type) { return aligned(p, type == NVFP4MOE_F32 ? 4 : 2); }

int spread(const void* token, int64_t ldt, int type, int64_t T, int64_t K, int k, const int32_t* f2p,
           const float* w, const void* dot_rows, int64_t ldd, void* rows, int64_t n_rows, int64_t ldr, float* d_w,
           void* stream) {
  NVFP4_TRY(check_sizes(type, T, K, k, n_rows));
  if (T == 0) return NVFP4MOE_OK;
  NVFP4_CHECK(f2p && (d_w ? w && (dot_rows || n_rows == 0 || K == 0) : !dot_rows), NVFP4MOE_ERR_INVALID);
  // (a token's row is read before its slots, of which all may be dropped)
  NVFP4_CHECK(K == 0 || (token && (n_rows == 0 || rows)), NVFP4MOE_ERR_INVALID);
  NVFP4_CHECK(ldt >= K && ldr >= K && (!dot_rows || ldd >= K), NVFP4MOE_ERR_INVALID);
  NVFP4_CHECK(element_aligned(token, type) && element_aligned(rows, type) && element_aligned(dot_rows, type),
              NVFP4MOE_ERR_INVALID);
  if (K == 0 && !d_w) return NVFP4MOE_OK;
  Args a{};
  a.token_in = token; a.ldt_in = ldt;
  a.rows_in = dot_rows; a.ldr_in = ldd;
  a.rows_out = rows; a.ldr_out = ldr;
  a.n_rows = n_rows; a.f2p = f2p; a.w = w; a.d_w = d_w; a.T = T; a.K = K; a.k = k;
  return launch(a, type, true, d_w != nullptr, stream);
}

int collect(const void* rows, int64_t n_rows, int64_t ldr, int type, int64_t T, int64_t K, int k,
            const int32_t* f2p, const float* w, const void* dot_token, int64_t ldd, void* token, int64_t ldt,
            float* d_w, void* stream) {
  NVFP4_TRY(check_sizes(type, T, K, k, n_rows));
  if (T == 0) return NVFP4MOE_OK;
  NVFP4_CHECK(f2p && (d_w ? w && (dot_token || K == 0) : !dot_token), NVFP4MOE_ERR_INVALID);
  NVFP4_CHECK(K == 0 || (token && (n_rows == 0 || rows)), NVFP4MOE_ERR_INVALID);
  NVFP4_CHECK(ldt >= K && ldr >= K && (!dot_token || ldd >= K), NVFP4MOE_ERR_INVALID);
  NVFP4_CHECK(element_aligned(token, type) && element_aligned(rows, type) && element_aligned(dot_token, type),
              NVFP4MOE_ERR_INVALID);
  if (K == 0 && !d_w) return NVFP4MOE_OK;
  Args a{};
  a.token_in = dot_token; a.ldt_in = ldd;
  a.token_out = token; a.ldt_out = ldt;
  a.rows_in = rows; a.ldr_in = ldr;
  a.n_rows = n_rows; a.f2p = f2p; a.w = w; a.d_w = d_w; a.T = T; a.K = K; a.k = k;
  return launch(a, type, false, d_w != nullptr, stream);
}

}  // namespace
}  // namespace nvfp4moe

using namespace nvfp4moe;

extern "C" int moe_sort_tokens(const void* x, int type, int64_t T, int64_t K, int64_t ldx,
                               const int32_t* flat_to_perm, int k, const float* topk_w, void* rows, int64_t n_rows,
                               int64_t ldr, void* stream) {
  return spread(x, ldx, type, T, K, k, flat_to_perm, topk_w, nullptr, 0, rows, n_rows, ldr, nullptr, stream);
}

extern "C" int moe_sort_tokens_backward(const void* d_rows, int type, int64_t n_rows, int64_t K, int64_t ldr,
                                        const int32_t* flat_to_perm, int64_t T, int k, const float* topk_w,
                                        const void* x, int64_t ldx, void* dx, int64_t lddx, float* d_w,
                                        void* stream) {
  return collect(d_rows, n_rows, ldr, type, T, K, k, flat_to_perm, topk_w, x, ldx, dx, lddx, d_w, stream);
}

extern "C" int moe_unsort_tokens(const void* rows, int type, int64_t n_rows, int64_t K, int64_t ldr,
                                 const int32_t* flat_to_perm, int64_t T, int k, const float* topk_w, void* y,
                                 int64_t ldy, void* stream) {
  return collect(rows, n_rows, ldr, type, T, K, k, flat_to_perm, topk_w, nullptr, 0, y, ldy, nullptr, stream);
}

extern "C" int moe_unsort_tokens_backward(const void* dy, int type, int64_t T, int64_t K, int64_t lddy,
                                          const int32_t* flat_to_perm, int k, const float* topk_w, const void* rows,
                                          int64_t ldr, void* d_rows, int64_t n_rows, int64_t lddr, float* d_w,
                                          void* stream) {
  return spread(dy, lddy, type, T, K, k, flat_to_perm, topk_w, rows, ldr, d_rows, n_rows, lddr, d_w, stream);
}
