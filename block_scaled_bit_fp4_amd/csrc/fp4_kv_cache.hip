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
// per token and head (2.28 times less out than in for BF16 NVFP4).  A lane
// owns one block (16 or 32 elements: 32 to 128 bytes in, 8 or 16 out), so a
// scale needs no exchange between lanes and every access is 16 bytes wide;
// consecutive lanes take consecutive blocks of a token, whole 2 * D byte
// rows of the input.
#include "fp4_kv.h"
#include "fp4_quantize.h"

using namespace fp4kv;

namespace {

struct AppendArgs {
  KvCacheArgs c;
  KvBatchArgs b;
  const void* x[2];       // K, V
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

// Unit u of a sequence's new tokens: token, K or V, head, block of the row.
struct Unit {
  int token, part, head, block;
  __device__ __forceinline__ Unit(uint32_t u, uint32_t heads, uint32_t blocks) {
    const uint32_t row = u / blocks;
    block = (int)(u - row * blocks);
    const uint32_t kv = row / heads;
    head = (int)(row - kv * heads);
    token = (int)(kv >> 1);
    part = (int)(kv & 1);
  }
};

template <int FMT, bool RHT, typename T>
__global__ __launch_bounds__(kThreads) void kv_append_kernel(AppendArgs a) {
  constexpr int B = block_of<FMT>();
  const int seq = blockIdx.y;
  const KvSeq sq = kv_seq(a.b, seq, a.c.page_log2);
  const uint32_t blocks = a.c.dim / B;
  const uint32_t per_token = 2u * a.c.heads * blocks;
  const uint32_t u = blockIdx.x * (uint32_t)kThreads + threadIdx.x;
  const Unit at(u, a.c.heads, blocks);
  if ((uint64_t)u >= (uint64_t)sq.n * per_token) return;
  const int64_t pos = sq.pos + at.token;
  if (pos < 0 || pos >= sq.kv) return;
  const int64_t row = row_of(a.c, a.b, seq, (int)pos, at.head);
  if (row < 0) return;
  const T* x = (at.part ? static_cast<const T*>(a.x[1]) : static_cast<const T*>(a.x[0])) +
               (sq.first + at.token) * (at.part ? a.token[1] : a.token[0]) +
               at.head * (at.part ? a.head[1] : a.head[0]) + at.block * B;
  RowRaw<T, B> raw;
  raw.load(x);
  float t[B], amax = 0.0f;
#pragma unroll
  for (int g = 0; g < B / 16; ++g) {
    float w[16];
    raw.template group<RHT>(g, w, a.c.signs);
    if constexpr (RHT) fwht16(w);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      t[16 * g + j] = w[j];
      amax = fmaxf(amax, fabsf(w[j]));
    }
  }
  ScaleCtx ctx{0.0f, 0.0f, 0.0f};
  if constexpr (FMT == kNVFP4) {
    ctx.s_t = at.part ? *a.c.v_scale : *a.c.k_scale;
    ctx.den = ctx.s_t * grid_max<FMT>();
  }
  uint32_t packed[B / 8], sbyte;
  encode_block<FMT, false, RHT, sizeof(T) == 2, B, kTsOuter>(t, amax, ctx, nullptr, 0u, 0u, 0u,
                                                             packed, sbyte);
  uint8_t* codes = (at.part ? a.c.v_codes : a.c.k_codes) + row * (a.c.dim / 2) + at.block * (B / 2);
  if constexpr (B == 16) store8<false>(codes, packed[0], packed[1]);
  else store16<false>(codes, packed[0], packed[1], packed[2], packed[3]);
  ((at.part ? a.c.v_scales : a.c.k_scales))[row * blocks + at.block] = (uint8_t)sbyte;
}

struct GatherArgs {
  KvCacheArgs c;
  KvBatchArgs b;
  void* out[2];
  int64_t token, head;
};

__device__ __forceinline__ void store_group(float* p, const float (&t)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    store16<false>(p + 4 * i, __float_as_uint(t[4 * i]), __float_as_uint(t[4 * i + 1]),
                   __float_as_uint(t[4 * i + 2]), __float_as_uint(t[4 * i + 3]));
}

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ void store_group(uint16_t* p, const float (&t)[16]) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const f32x2 v = {t[2 * i], t[2 * i + 1]};
    w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
  }
  store16<false>(p, w[0], w[1], w[2], w[3]);
  store16<false>(p + 8, w[4], w[5], w[6], w[7]);
}

// A lane reads one 16-element group: eight code bytes and its block's scale.
template <int B, typename T>
__global__ __launch_bounds__(kThreads) void kv_gather_kernel(GatherArgs a) {
  const int seq = blockIdx.y;
  const KvSeq sq = kv_seq(a.b, seq, a.c.page_log2);
  const uint32_t groups = a.c.dim / 16;
  const uint32_t u = blockIdx.x * (uint32_t)kThreads + threadIdx.x;
  const Unit at(u, a.c.heads, groups);
  if ((uint64_t)u >= (uint64_t)sq.n * (2u * a.c.heads * groups)) return;
  const int64_t pos = sq.pos + at.token;
  const int64_t row =
      pos < 0 || pos >= sq.kv ? -1 : row_of(a.c, a.b, seq, (int)pos, at.head);
  float t[16];
  if (row < 0) {  // no such token in the cache: zeros
#pragma unroll
    for (int j = 0; j < 16; ++j) t[j] = 0.0f;
  } else {
    const uint2 w = *reinterpret_cast<const uint2*>((at.part ? a.c.v_codes : a.c.k_codes) +
                                                    row * (a.c.dim / 2) + at.block * 8);
    const uint32_t S = (at.part ? a.c.v_scales : a.c.k_scales)[row * (a.c.dim / B) +
                                                               at.block * 16 / B];
    float d;
    if constexpr (B == 16) d = (at.part ? *a.c.v_scale : *a.c.k_scale) * e4m3_decode(S);
    else d = S ? __uint_as_float(S << 23) : 0x1p-127f;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const uint32_t c = ((j < 8 ? w.x : w.y) >> (4 * (j & 7))) & 15u;
      const float v = e2m1_level(c & 7u) * d;
      t[j] = (c & 8u) ? -v : v;
    }
    if (a.c.rht) rht16_inverse(t, a.c.signs);
  }
  T* out = static_cast<T*>(at.part ? a.out[1] : a.out[0]) + (sq.first + at.token) * a.token +
           at.head * a.head + at.block * 16;
  store_group(out, t);
}

template <int FMT, bool RHT>
hipError_t launch_append(const AppendArgs& a, int dtype, dim3 grid, hipStream_t s) {
  if (dtype == 0) kv_append_kernel<FMT, RHT, uint16_t><<<grid, kThreads, 0, s>>>(a);
  else kv_append_kernel<FMT, RHT, float><<<grid, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t fp4_launch_kv_append(const KvAppendLaunch& q, hipStream_t s) {
  AppendArgs a{};
  a.c = q.cache;
  a.b = q.batch;
  a.x[0] = q.k;
  a.x[1] = q.v;
  a.token[0] = q.k_token;
  a.token[1] = q.v_token;
  a.head[0] = q.k_head;
  a.head[1] = q.v_head;
  const int B = q.cache.format == kNVFP4 ? 16 : 32;
  const int64_t units = (int64_t)q.batch.max_q * 2 * q.cache.heads * (q.cache.dim / B);
  const dim3 grid((unsigned)((units + kThreads - 1) / kThreads), (unsigned)q.batch.batch);
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
  GatherArgs a{};
  a.c = q.cache;
  a.b = q.batch;
  a.out[0] = q.k;
  a.out[1] = q.v;
  a.token = q.token;
  a.head = q.head;
  const int64_t units = (int64_t)q.batch.max_q * 2 * q.cache.heads * (q.cache.dim / 16);
  const dim3 grid((unsigned)((units + kThreads - 1) / kThreads), (unsigned)q.batch.batch);
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
