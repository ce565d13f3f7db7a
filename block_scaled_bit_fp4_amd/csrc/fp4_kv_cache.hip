// fp4_kv_cache.hip -- writing new K and V rows into the pages of a 4-bit
// cache, and reading them back.
//
// Write: y = RHT(x) per 16-group of a head's row (optional), then block
// scales and codes exactly as fp4_quantize's row axis gives them with a
// given tensor scale (encode_block is the same code), stored at the token's
// place instead of row-major.  K and V go in one launch.  Read: L[k] * d,
// one binary32 product, then the inverse RHT.
//
// Bound by bytes: 2 * D * element size read and 2 * (D / 2 + D / B) written
// per token and head (2.28 times less out than in for BF16 NVFP4), or the
// reverse.  Writing takes 32 bytes of a row in a lane, reading back gives 16:
// consecutive lanes touch consecutive bytes, and a block or 16-group that
// lies in two or four lanes is joined by DPP moves.  (A whole block to a
// lane strides 128 bytes between lanes for FP32.)  A lane has a few pieces in
// flight, so that the chain length -> page -> data is waited for once, and
// what is not used again goes past the caches.  A piece's place is found once
// and the division by the heads is a product: reading back was bound by the
// vector unit before (105 us for what now takes 73).
//
// 51535 tokens of eight FP32 heads of 128 columns (MXFP4: 0.48 GB each way)
// take 94 us to write (5.1 TB/s) and 73 us to read back (6.5); with a lane to
// a block 126 and 150.  Writing with each lane's 32 bytes loaded in place (two
// loads that touch every other 16 bytes) took 105 us, 122 without the
// non-temporal loads; runs of neighbouring tokens kept on one chiplet change
// nothing.
#include "fp4_kv.h"
#include "fp4_quantize.h"

#include <type_traits>

using namespace fp4kv;

namespace {

// Pieces of a lane, at once.  Writing (before the loads were swapped between
// lanes): 113, 105, 109, 105 us for one to four; reading back: 84, 72, 74, 73
// for two, four, six, eight.  (Single tokens: 3.5 to 3.9 and 3.2 to 4.2 us.)
constexpr int kAppendPieces = 2, kGatherPieces = 4;

// Division by the number of heads d: n / d = (n * m >> 32) >> s for n < 2^31,
// with s = ceil(log2 d) - 1 and m = floor(2^(32 + s) / d) + 1.  With e = m d -
// 2^(32 + s), 0 < e <= d <= 2^(s + 1): n m / 2^(32 + s) = n / d + n e / (d
// 2^(32 + s)), whose last term is below 1 / d, so the floor is that of n / d.
struct Heads {
  uint32_t d, m;
  int s;
  explicit Heads(uint32_t heads) : d(heads), m(0), s(0) {
    while ((2u << s) < d) ++s;
    m = (uint32_t)((1ull << (32 + s)) / d + 1);
  }
  __device__ __forceinline__ uint32_t under(uint32_t n) const { return d == 1 ? n : __umulhi(n, m) >> s; }
};

struct AppendArgs {
  KvCacheArgs c;
  KvBatchArgs b;
  Heads heads;
  const void* x[2];  // K, V
  int64_t token[2], head[2];
};

// Place of position `pos` of sequence `seq`, as a row of the layer's
// [pages][heads][page] rows for head h; -1 if the sequence has no page there.
__device__ __forceinline__ int64_t row_of(const KvCacheArgs& c, const KvBatchArgs& b, int seq,
                                          int pos, int h) {
  const int page = b.page_table[seq * b.table_ld + (pos >> c.page_log2)];
  if (page < 0 || page >= c.pages) return -1;
  return (((int64_t)page * c.heads + h) << c.page_log2) + (pos & ((1 << c.page_log2) - 1));
}

// Unit u of a sequence's new tokens: token, K or V, head, piece of the row
// (1 << log2 pieces).
struct Unit {
  int token, part, head, piece;
  __device__ __forceinline__ Unit(uint32_t u, const Heads& heads, int log2) {
    const uint32_t row = u >> log2;
    piece = (int)(u & ((1u << log2) - 1));
    const uint32_t kv = heads.under(row);
    head = (int)(row - kv * heads.d);
    token = (int)(kv >> 1);
    part = (int)(kv & 1);
  }
};

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __uint_as_float(
      (uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, 0xF, 0xF, true));
}

// The value of the lane that is STEP (1, 2 or 4) away, lane ^ STEP.
template <int STEP>
__device__ __forceinline__ float neighbour(float v) {
  if constexpr (STEP == 1) return dpp<0xB1>(v);  // quad_perm [1 0 3 2]
  else if constexpr (STEP == 2) return dpp<0x4E>(v);  // quad_perm [2 3 0 1]
  else {
    const float up = dpp<0x104>(v), down = dpp<0x114>(v);  // row_shl 4, row_shr 4
    return threadIdx.x & 4 ? down : up;
  }
}

// The 16-point transform of a group that lies E elements to a lane, in lanes
// L apart, in the order of fwht16 (steps 1, 2, 4, 8: the same sums).  at: the
// lane's first element.
template <int L, int E>
__device__ __forceinline__ void fwht_lanes(float (&t)[E], int at) {
#pragma unroll
  for (int h = 1; h < E && h < 16; h <<= 1)
#pragma unroll
    for (int j = 0; j < E; ++j) {
      if (j & h) continue;
      const float u = t[j], v = t[j + h];
      t[j] = u + v;
      t[j + h] = u - v;
    }
  if constexpr (E < 16) {
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const float o = neighbour<L>(t[j]);
      t[j] = at & E ? o - t[j] : t[j] + o;
    }
  }
  if constexpr (E < 8) {
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const float o = neighbour<2 * L>(t[j]);
      t[j] = at & (2 * E) ? o - t[j] : t[j] + o;
    }
  }
}

template <int E>
__device__ __forceinline__ void signs_of(float (&t)[E], uint32_t signs, int at) {
#pragma unroll
  for (int j = 0; j < E; ++j)
    t[j] = __uint_as_float(__float_as_uint(t[j]) ^ ((signs >> ((at + j) & 15)) << 31));
}

typedef uint32_t u4 __attribute__((ext_vector_type(4)));

template <int FMT, bool RHT, typename T>
__global__ __launch_bounds__(kThreads) void kv_append_kernel(AppendArgs a) {
  constexpr int B = block_of<FMT>();
  constexpr int E = 32 / sizeof(T);  // elements of a piece
  constexpr int kLog2 = E == 16 ? 4 : 3;
  const int seq = blockIdx.y;
  const KvSeq sq = kv_seq(a.b, seq, a.c.page_log2);
  const int pieces_log2 = a.c.dim_log2 - kLog2;
  const uint32_t units = (uint32_t)sq.n * 2u * a.c.heads << pieces_log2;
  const uint32_t first = blockIdx.x * (uint32_t)(kThreads * kAppendPieces) + threadIdx.x;
  if (first - threadIdx.x >= units) return;
  // A wave's 64 pieces of 32 bytes are loaded as two runs of 1024, sixteen
  // bytes to a lane; lane pairs then swap halves, so that the even lanes have
  // the pieces of the first run and the odd ones those of the second.
  u4 raw[kAppendPieces][2];
  int64_t row[kAppendPieces];
  int part[kAppendPieces], at_in[kAppendPieces];
  const bool odd = threadIdx.x & 1;
#pragma unroll
  for (int k = 0; k < kAppendPieces; ++k) {
    const uint32_t u = (first & ~63u) + k * kThreads + (threadIdx.x & 63) / 2;
    const Unit a0(u < units ? u : 0u, a.heads, pieces_log2);
    const Unit a1(u + 32 < units ? u + 32 : 0u, a.heads, pieces_log2);
    auto load = [&](const Unit& at) {
      const T* x = (at.part ? static_cast<const T*>(a.x[1]) : static_cast<const T*>(a.x[0])) +
                   (sq.first + at.token) * (at.part ? a.token[1] : a.token[0]) +
                   at.head * (at.part ? a.head[1] : a.head[0]) + at.piece * E;
      return __builtin_nontemporal_load(reinterpret_cast<const u4*>(x) + (odd ? 1 : 0));
    };
    raw[k][0] = load(a0);
    raw[k][1] = load(a1);
    const int64_t pos = sq.pos + (odd ? a1.token : a0.token);
    part[k] = odd ? a1.part : a0.part;
    at_in[k] = (odd ? a1.piece : a0.piece) * E;
    row[k] = (odd ? u + 32 : u) < units && pos >= 0 && pos < sq.kv
                 ? row_of(a.c, a.b, seq, (int)pos, odd ? a1.head : a0.head)
                 : -1;
  }
#pragma unroll
  for (int k = 0; k < kAppendPieces; ++k) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t give = odd ? raw[k][0][e] : raw[k][1][e];
      const uint32_t get = __float_as_uint(neighbour<1>(__uint_as_float(give)));
      raw[k][0][e] = odd ? get : raw[k][0][e];
      raw[k][1][e] = odd ? raw[k][1][e] : get;
    }
  }
#pragma unroll
  for (int k = 0; k < kAppendPieces; ++k) {
    // lanes of a block (and of a 16-group) take the same way
    if (row[k] < 0) continue;
    float t[E], amax = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t w = raw[k][j / 4][j % 4];
      if constexpr (E == 16) {
        t[2 * j] = __uint_as_float(w << 16);
        t[2 * j + 1] = __uint_as_float(w & 0xFFFF0000u);
      } else {
        t[j] = __uint_as_float(w);
      }
    }
    if constexpr (RHT) {
      signs_of(t, a.c.signs, at_in[k]);
      fwht_lanes<2>(t, at_in[k]);
    }
#pragma unroll
    for (int j = 0; j < E; ++j) amax = fmaxf(amax, fabsf(t[j]));
    if constexpr (B > E) amax = fmaxf(amax, neighbour<2>(amax));
    if constexpr (B > 2 * E) amax = fmaxf(amax, neighbour<4>(amax));
    ScaleCtx ctx{0.0f, 0.0f, 0.0f};
    if constexpr (FMT == kNVFP4) {
      ctx.s_t = part[k] ? *a.c.v_scale : *a.c.k_scale;
      ctx.den = ctx.s_t * grid_max<FMT>();
    }
    uint32_t packed[E / 8], sbyte;
    encode_block<FMT, false, RHT, sizeof(T) == 2, E, kTsOuter>(t, amax, ctx, nullptr, 0u, 0u, 0u,
                                                               packed, sbyte);
    uint8_t* codes = (part[k] ? a.c.v_codes : a.c.k_codes) + (row[k] << (a.c.dim_log2 - 1)) +
                     at_in[k] / 2;
    if constexpr (E == 16) store8<false>(codes, packed[0], packed[1]);
    else *reinterpret_cast<uint32_t*>(codes) = packed[0];
    if (at_in[k] % B == 0)
      (part[k] ? a.c.v_scales : a.c.k_scales)[row[k] * (a.c.dim / B) + at_in[k] / B] =
          (uint8_t)sbyte;
  }
}

struct GatherArgs {
  KvCacheArgs c;
  KvBatchArgs b;
  Heads heads;
  void* out[2];
  int64_t token, head;
};

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ u4 out_of(const float (&t)[4]) {
  return u4{__float_as_uint(t[0]), __float_as_uint(t[1]), __float_as_uint(t[2]),
            __float_as_uint(t[3])};
}
__device__ __forceinline__ u4 out_of(const float (&t)[8]) {
  u4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f32x2 v = {t[2 * i], t[2 * i + 1]};
    w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
  }
  return w;
}

// Levels of E codes.
template <int E>
__device__ __forceinline__ void levels(uint32_t codes, float (&t)[E]) {
  auto two = [&](auto byte) {
    const f32x2 v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, decltype(byte)::value);
    t[2 * decltype(byte)::value] = v.x;
    t[2 * decltype(byte)::value + 1] = v.y;
  };
  two(std::integral_constant<int, 0>{});
  two(std::integral_constant<int, 1>{});
  if constexpr (E == 8) {
    two(std::integral_constant<int, 2>{});
    two(std::integral_constant<int, 3>{});
  }
}

template <int B, typename T>
__global__ __launch_bounds__(kThreads) void kv_gather_kernel(GatherArgs a) {
  constexpr int E = 16 / sizeof(T);  // elements of a piece
  constexpr int kLog2 = E == 8 ? 3 : 2;
  typedef typename std::conditional<E == 8, uint32_t, uint16_t>::type codes_t;
  const int seq = blockIdx.y;
  const KvSeq sq = kv_seq(a.b, seq, a.c.page_log2);
  const int pieces_log2 = a.c.dim_log2 - kLog2;
  const uint32_t units = (uint32_t)sq.n * 2u * a.c.heads << pieces_log2;
  const uint32_t first = blockIdx.x * (uint32_t)(kThreads * kGatherPieces) + threadIdx.x;
  if (first - threadIdx.x >= units) return;
  uint32_t codes[kGatherPieces], scale[kGatherPieces];
  T* out[kGatherPieces];
  int part[kGatherPieces];
  bool held[kGatherPieces];
  const int at_in = (threadIdx.x & ((1 << pieces_log2) - 1)) * E;  // the same for all pieces
#pragma unroll
  for (int k = 0; k < kGatherPieces; ++k) {
    const uint32_t u = first + k * kThreads;
    const Unit at(u < units ? u : 0u, a.heads, pieces_log2);
    const int64_t pos = sq.pos + at.token;
    int64_t row = u < units && pos >= 0 && pos < sq.kv ? row_of(a.c, a.b, seq, (int)pos, at.head) : -1;
    held[k] = row >= 0;
    if (row < 0) row = 0;
    part[k] = at.part;
    out[k] = static_cast<T*>(at.part ? a.out[1] : a.out[0]) + (sq.first + at.token) * a.token +
             at.head * a.head + at_in;
    codes[k] = *reinterpret_cast<const codes_t*>((at.part ? a.c.v_codes : a.c.k_codes) +
                                                 (row << (a.c.dim_log2 - 1)) + at_in / 2);
    scale[k] = (at.part ? a.c.v_scales : a.c.k_scales)[row * (a.c.dim / B) + at_in / B];
  }
#pragma unroll
  for (int k = 0; k < kGatherPieces; ++k) {
    if (first + k * kThreads >= units) return;  // whole rows: lanes of a 16-group take the same way
    float d;
    if constexpr (B == 16) d = (part[k] ? *a.c.v_scale : *a.c.k_scale) * e4m3_decode(scale[k]);
    else d = scale[k] ? __uint_as_float(scale[k] << 23) : 0x1p-127f;
    if (!held[k]) {  // no such token in the cache
      codes[k] = 0;
      d = 0.0f;
    }
    float t[E];
    levels(codes[k], t);
#pragma unroll
    for (int j = 0; j < E; ++j) t[j] *= d;
    if (a.c.rht) {
      fwht_lanes<1>(t, at_in);
#pragma unroll
      for (int j = 0; j < E; ++j) t[j] *= 0.25f;
      signs_of(t, held[k] ? a.c.signs : 0u, at_in);
    }
    __builtin_nontemporal_store(out_of(t), reinterpret_cast<u4*>(out[k]));
  }
}

template <int FMT, bool RHT>
hipError_t launch_append(const AppendArgs& a, int dtype, dim3 grid, hipStream_t s) {
  if (dtype == 0) kv_append_kernel<FMT, RHT, uint16_t><<<grid, kThreads, 0, s>>>(a);
  else kv_append_kernel<FMT, RHT, float><<<grid, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

// Workgroups for the longest sequence's new tokens, in lanes of `pieces` of
// `elements` each, and for all sequences.
dim3 grid_of(const KvCacheArgs& c, const KvBatchArgs& b, int elements, int pieces) {
  const int64_t units = (int64_t)b.max_q * 2 * c.heads * (c.dim / elements), n = kThreads * pieces;
  return dim3((unsigned)((units + n - 1) / n), (unsigned)b.batch);
}

}  // namespace

hipError_t fp4_launch_kv_append(const KvAppendLaunch& q, hipStream_t s) {
  AppendArgs a{q.cache, q.batch, Heads(q.cache.heads), {}, {}, {}};
  a.x[0] = q.k;
  a.x[1] = q.v;
  a.token[0] = q.k_token;
  a.token[1] = q.v_token;
  a.head[0] = q.k_head;
  a.head[1] = q.v_head;
  const dim3 grid = grid_of(q.cache, q.batch, q.dtype == 0 ? 16 : 8, kAppendPieces);
  switch (q.cache.format) {
    case kNVFP4:
      return q.cache.rht ? launch_append<kNVFP4, true>(a, q.dtype, grid, s)
                         : launch_append<kNVFP4, false>(a, q.dtype, grid, s);
    case kMXFP4:
      return q.cache.rht ? launch_append<kMXFP4, true>(a, q.dtype, grid, s)
                         : launch_append<kMXFP4, false>(a, q.dtype, grid, s);
    default:
      return q.cache.rht ? launch_append<kMXOAS, true>(a, q.dtype, grid, s)
                         : launch_append<kMXOAS, false>(a, q.dtype, grid, s);
  }
}

hipError_t fp4_launch_kv_gather(const KvGatherLaunch& q, hipStream_t s) {
  GatherArgs a{q.cache, q.batch, Heads(q.cache.heads), {}, 0, 0};
  a.out[0] = q.k;
  a.out[1] = q.v;
  a.token = q.token;
  a.head = q.head;
  const dim3 grid = grid_of(q.cache, q.batch, q.dtype == 0 ? 8 : 4, kGatherPieces);
  const bool nv = q.cache.format == kNVFP4;
  if (q.dtype == 0) {
    if (nv) kv_gather_kernel<16, uint16_t><<<grid, kThreads, 0, s>>>(a);
    else kv_gather_kernel<32, uint16_t><<<grid, kThreads, 0, s>>>(a);
  } else {
    if (nv) kv_gather_kernel<16, float><<<grid, kThreads, 0, s>>>(a);
    else kv_gather_kernel<32, float><<<grid, kThreads, 0, s>>>(a);
  }
  return hipGetLastError();
}
