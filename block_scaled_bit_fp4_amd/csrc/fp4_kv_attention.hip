// fp4_kv_attention.hip -- attention of new tokens over a 4-bit paged cache.
//
// For each new token t at position p and query head (H query heads share
// the G = H / heads keys' head): s_j = scale * <q, K_j> over the visible
// positions j <= p (under a window: j > p - window, or j < sinks), o = sum_j
// exp(s_j - m) V_j / sum_j exp(s_j - m), lse = m + log of that sum.  A cache
// of rotated rows holds K H and V H (H the orthogonal 16-point transform), so
// q is rotated too, <q H, K H> = <q, K>, and o is rotated back; codes and
// scales are never rotated.
//
// Number types.  An E2M1 level has 2 significant bits and an E4M3 scale 4,
// so level * scale has at most 6 bits and lies in [2^-10, 2688]: exact in
// FP16, NVFP4 runs on FP16 matrix instructions with the layer's factor
// applied to the scores and the output in 32 bits.  q goes to FP16 after an
// exact power-of-two scaling of its row to [1, 2) at its largest element
// (BF16's 8 bits fit; a rotated q rounds at 2^-12).  An E8M0 scale spans the
// exponents of binary32, so MXFP4 runs on BF16, where level * 2^e is exact;
// a rotated q, which BF16 would round at 2^-9, is split into two BF16 parts
// whose products are both taken.  Probabilities round to the same 16-bit
// type (2^-12 or 2^-9, relative to the running maximum), and the row sum
// adds the rounded values, so that an error in a large one cancels.  Scores,
// maxima, sums and outputs are held in 32 bits.
//
// Products are taken as S^T = K q^T and O^T = V^T P^T.  An instruction
// leaves S^T with the row's query in the lane and four consecutive keys in
// its registers; P^T wants a lane's query and eight keys of its own choice
// (any order of the contraction serves if V^T follows it), so P needs no move
// between lanes.  V comes row by row (a token's 4-bit row is what is stored)
// and is wanted column by column: the dequantized rows go to LDS and come
// back through the 16-bit transposing read (a group of 16 lanes reads 4 rows
// of 16 values, lane i gets column i).
#include "fp4_device.h"
#include "fp4_kv.h"

using namespace fp4dev;
using namespace fp4kv;

namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t w2 __attribute__((ext_vector_type(2)));
typedef uint32_t w4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// The 16-bit type of a format's products.
template <bool MX>
struct Num;
template <>
struct Num<false> {
  typedef _Float16 x2 __attribute__((ext_vector_type(2)));
  typedef _Float16 x8 __attribute__((ext_vector_type(8)));
  static __device__ __forceinline__ f32x4 mma(x8 a, x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x16 mma(x8 a, x8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
  }
  static constexpr uint32_t kOnes = 0x3C003C00u;
};
template <>
struct Num<true> {
  typedef __bf16 x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 x8 __attribute__((ext_vector_type(8)));
  static __device__ __forceinline__ f32x4 mma(x8 a, x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x16 mma(x8 a, x8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
  static constexpr uint32_t kOnes = 0x3F803F80u;
};

// Two floats rounded to the 16-bit type (to nearest, ties to even).
template <bool MX>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const f32x2 v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, typename Num<MX>::x2));
}

template <bool MX>
__device__ __forceinline__ typename Num<MX>::x8 as8(const w4& w) {
  return __builtin_bit_cast(typename Num<MX>::x8, w);
}

// Eight codes (one word, element 0 in the low nibble) to eight values.  NVFP4:
// the pair convert gives the levels, a packed FP16 product applies the scale
// (exact).  MX: the convert applies the power-of-two scale itself.
template <bool MX>
struct Scale;  // the scale of a run of codes
template <>
struct Scale<false> {
  Num<false>::x2 s;  // the same value twice
};
template <>
struct Scale<true> {
  float s;
};

__device__ __forceinline__ w4 dequant8(uint32_t w, const Scale<false>& k) {
  w4 r;
  r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0) * k.s);
  r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1) * k.s);
  r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2) * k.s);
  r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3) * k.s);
  return r;
}
__device__ __forceinline__ w4 dequant8(uint32_t w, const Scale<true>& k) {
  w4 r;
  r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, k.s, 0));
  r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, k.s, 1));
  r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, k.s, 2));
  r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, k.s, 3));
  return r;
}

// Scale of block i of a lane's scale bytes.  E8M0 byte b is 2^(b - 127); the
// convert reads the exponent field of its scale operand, so b << 23 serves
// for b = 0 too.
__device__ __forceinline__ void block_scale(uint32_t bytes, int i, Scale<false>& k) {
  const auto p = (i & 2) ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(bytes, 1.0f, true)
                         : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(bytes, 1.0f, false);
  k.s = (i & 1) ? __builtin_shufflevector(p, p, 1, 1) : __builtin_shufflevector(p, p, 0, 0);
}
__device__ __forceinline__ void block_scale(uint32_t bytes, int i, Scale<true>& k) {
  k.s = __uint_as_float(((bytes >> (8 * i)) & 0xFFu) << 23);
}

struct Args {
  KvCacheArgs c;
  KvBatchArgs b;
  const uint16_t* q;
  int64_t q_token, q_head;
  int q_heads, group;  // group: query heads of a key head
  float scale;
  int window, sinks;
  void* out;
  int out_f32;
  int64_t out_token, out_head;
  float* lse;
  // pieces of the keys: partial outputs [split][token][head][D], and (m, l)
  // of each [split][token][head]
  float* part;
  float2* part_ml;
  int splits, row_tiles;
};

// The keys that the rows of a workgroup see: the tiles of T keys that hold
// the first `sinks` tokens, then those from the first row's window to the
// last row's position, cut to this split.
template <int T>
struct Keys {
  int sink_tiles, start, begin, end;  // tiles [begin, end) of the list
  int lo, hi;                         // visible to some row: [lo, hi), and the sinks
  __device__ __forceinline__ void init(const Args& a, const KvSeq& s, int i0, int i1, int split) {
    const int64_t p0 = s.pos + i0, p1 = s.pos + i1;
    const int64_t h = p1 + 1 < s.kv ? p1 + 1 : s.kv;
    hi = h < 0 ? 0 : (int)h;
    lo = 0;
    if (a.window > 0 && p0 + 1 > a.window) lo = (int)(p0 + 1 - a.window < hi ? p0 + 1 - a.window : hi);
    const int sk = a.sinks < lo ? a.sinks : lo;
    sink_tiles = (sk + T - 1) / T;
    start = lo / T > sink_tiles ? lo / T : sink_tiles;
    const int last = (hi + T - 1) / T;
    const int n = sink_tiles + (last > start ? last - start : 0);
    // every split takes the same number of tiles whatever the sequence, so
    // that lengths apart leave workgroups of equal work (the host sizes the
    // splits by the longest list); a list past that bound is shared evenly
    const int bound = (max_keys(a, s) + T - 1) / T + 2;
    const int per = ((n > bound ? n : bound) + a.splits - 1) / a.splits;
    const int64_t b = (int64_t)split * per;
    begin = b < n ? (int)b : n;
    end = b + per < n ? (int)(b + per) : n;
  }
  // Most keys a row tile of this call sees, by what the host knows.
  static __device__ __forceinline__ int max_keys(const Args& a, const KvSeq& s) {
    int64_t n = a.b.max_kv;
    if (a.window > 0) {
      const int64_t w = (int64_t)a.window + a.sinks + a.b.max_q;
      if (w < n) n = w;
    }
    return (int)n;
  }
  __device__ __forceinline__ int base(int u) const {
    return (u < sink_tiles ? u : start + u - sink_tiles) * T;
  }
};

// Page of the sixteen tokens from t on (t a multiple of 16, wave-uniform),
// -1 if the sequence has none there.
__device__ __forceinline__ int page_of(const Args& a, int seq, int t, int hi) {
  if (t >= hi) return -1;
  const int p = a.b.page_table[seq * a.b.table_ld + (t >> a.c.page_log2)];
  return p >= 0 && p < a.c.pages ? p : -1;
}

__device__ __forceinline__ int64_t row_of(const Args& a, int page, int h, int t) {
  return (((int64_t)(page < 0 ? 0 : page) * a.c.heads + h) << a.c.page_log2) +
         (t & ((1 << a.c.page_log2) - 1));
}

// ------------------------------------------------------------ q's fragments
// Elements d0 .. d0 + 16 of a row of q, rotated if the cache's rows are.
__device__ __forceinline__ void load_q16(const uint16_t* p, bool rht, uint32_t signs,
                                         float (&t)[16]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p), b = *reinterpret_cast<const uint4*>(p + 8);
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  widen_bf16_group<false>(w, 0u, t);
  if (rht) rht16_forward(t, signs);
}

// 2^-e and 2^e for the largest magnitude m = 1.f * 2^e of a row, kept to
// exponents whose powers are normal; 1 for a row of zeros.
__device__ __forceinline__ void row_power(float m, float& down, float& up) {
  int e = (int)(__float_as_uint(m) >> 23);
  e = m > 0.0f ? (e < 2 ? 2 : (e > 252 ? 252 : e)) : 127;
  down = __uint_as_float((uint32_t)(254 - e) << 23);
  up = __uint_as_float((uint32_t)e << 23);
}

// Scores are scaled by this in the base-2 exponent: |scale| * log2(e) and,
// for NVFP4, the layer's factor and the power taken out of the row of q.
// At least the smallest normal number, so that a masked score (-inf) stays
// -inf under it.
template <bool MX>
__device__ __forceinline__ float score_scale(const Args& a, float up) {
  float s = fabsf(a.scale) * 1.4426950408889634f;
  if constexpr (!MX) s = s * (fabsf(*a.c.k_scale) * up);
  return fmaxf(s, 0x1p-126f);
}
template <bool MX>
__device__ __forceinline__ float score_sign(const Args& a) {
  bool neg = a.scale < 0.0f;
  if constexpr (!MX) neg = neg != (*a.c.k_scale < 0.0f);
  return neg ? -1.0f : 1.0f;
}

// ------------------------------------------------------------------ outputs
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  const f32x2 v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

// Sixteen final values of one row of the output.
__device__ __forceinline__ void store_out16(const Args& a, int64_t token, int head, int d0,
                                            const float (&t)[16]) {
  const int64_t at = token * a.out_token + head * a.out_head + d0;
  if (a.out_f32) {
    f32x4* p = reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = f32x4{t[4 * i], t[4 * i + 1], t[4 * i + 2], t[4 * i + 3]};
  } else {
    w4* p = reinterpret_cast<w4*>(static_cast<uint16_t*>(a.out) + at);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      p[i] = w4{bf16_pair(t[8 * i], t[8 * i + 1]), bf16_pair(t[8 * i + 2], t[8 * i + 3]),
                bf16_pair(t[8 * i + 4], t[8 * i + 5]), bf16_pair(t[8 * i + 6], t[8 * i + 7])};
  }
}

// The factor that turns a row's sum of exp * level * scale into the output:
// one over the sum (0 where no key is visible) times the layer's factor.
template <bool MX>
__device__ __forceinline__ float out_factor(const Args& a, float l) {
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
  if constexpr (MX) return inv;
  else return inv * *a.c.v_scale;
}

__device__ __forceinline__ float row_lse(float m, float l) {
  return l > 0.0f ? (m + __builtin_amdgcn_logf(l)) * 0.69314718055994531f : -__builtin_inff();
}

// ============================================================ few new tokens
// Rows (a new token and a query head of this key head) 16 * NT to a
// workgroup of four waves.  Each wave takes every fourth tile of 32 keys of
// the split on its own: K's codes go from global memory through registers
// into the matrix instruction (a lane holds D / 4 codes of one token), V's
// through the wave's own LDS.  No barrier until the four waves' results are
// joined.
constexpr int kFewThreads = 256, kFewWaves = 4, kFewKeys = 32;

template <bool MX, int D>
struct FewTile {
  static constexpr int W = D / 32;  // words of codes per lane and row
  uint32_t k[2][W], v[2][W];
  uint32_t ks[2], vs[2];
  int page[2];
};

template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N == 2) {
    const w2 t = *reinterpret_cast<const w2*>(p);
    w[0] = t.x; w[1] = t.y;
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const w4 t = reinterpret_cast<const w4*>(p)[i];
      w[4 * i] = t.x; w[4 * i + 1] = t.y; w[4 * i + 2] = t.z; w[4 * i + 3] = t.w;
    }
  }
}

// The scale bytes of a lane's D / 4 codes (segment g of the row).
template <bool MX, int D>
__device__ __forceinline__ uint32_t load_scales(const uint8_t* row, int g) {
  if constexpr (MX) {
    if constexpr (D == 64) return row[g >> 1];
    else if constexpr (D == 128) return row[g];
    else return *reinterpret_cast<const uint16_t*>(row + 2 * g);
  } else {
    if constexpr (D == 64) return row[g];
    else if constexpr (D == 128) return *reinterpret_cast<const uint16_t*>(row + 2 * g);
    else return *reinterpret_cast<const uint32_t*>(row + 4 * g);
  }
}

// Codes of 8-code word j of a lane's run lie in its scale block:
template <bool MX>
__device__ __forceinline__ constexpr int block_of_word(int j) {
  return MX ? j / 4 : j / 2;
}

template <bool MX, int D>
__device__ __forceinline__ void few_load(const Args& a, int h, int t0, int hi, const int (&page)[2],
                                         FewTile<MX, D>& x) {
  constexpr int B = MX ? 32 : 16;
  const int m = threadIdx.x & 15, g = (threadIdx.x >> 4) & 3;
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    x.page[r] = page[r];
    // sixteen tokens lie in one page; a page that the sequence does not have
    // is read as page 0 and its tokens are masked
    const int64_t row = row_of(a, page[r], h, t0 + 16 * r) + m;
    load_words(a.c.k_codes + row * (D / 2) + g * (D / 8), x.k[r]);
    load_words(a.c.v_codes + row * (D / 2) + g * (D / 8), x.v[r]);
    x.ks[r] = load_scales<MX, D>(a.c.k_scales + row * (D / B), g);
    x.vs[r] = load_scales<MX, D>(a.c.v_scales + row * (D / B), g);
  }
}

// LDS place (bytes) of 16-byte piece p of row r of a wave's V tile: pieces
// XOR-ed by the row so that the sixteen rows of a store phase (one piece)
// and the eight rows of a transposing read's half wave (two pieces) reach
// distinct banks.
template <int D>
__device__ __forceinline__ int few_at(int r, int p) {
  const int s = D == 64 ? 2 * ((r >> 1) & 3) + ((r >> 3) & 1) : 2 * (r & 7) + ((r >> 3) & 1);
  return r * (2 * D) + ((p ^ s) << 4);
}

__device__ __forceinline__ w2 read_tr16(const uint8_t* p) {
  return __builtin_bit_cast(w2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                    (__attribute__((address_space(3))) s16x4*)p));
}

// LDS traffic of one wave with itself: keeps the compiler from moving LDS
// accesses across (the hardware keeps a wave's LDS accesses in order).
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Largest of the four lanes that hold one row's keys.
__device__ __forceinline__ float max_over_g(float v) {
  v = fmaxf(v, __shfl_xor(v, 16));
  return fmaxf(v, __shfl_xor(v, 32));
}

template <int D>
constexpr int few_lds() {
  constexpr int v = kFewWaves * kFewKeys * 2 * D;          // V tiles
  constexpr int o = kFewWaves * 16 * (D + 4) * 4 + 1024;   // joining: outputs, (m, l)
  return v > o ? v : o;
}

template <bool MX, bool LO, int D, int NT>
__global__ __launch_bounds__(kFewThreads, NT == 1 && D <= 128 ? 3 : 1) void kv_few_kernel(Args a) {
  typedef Num<MX> N;
  typedef typename N::x8 x8;
  constexpr int W = D / 32;  // words of codes per lane = QK instructions
  constexpr int J = D / 16;  // PV instructions (columns of 16)
  __shared__ __align__(16) uint8_t lds[few_lds<D>()];

  int id = blockIdx.x;
  const int split = id % a.splits;
  id /= a.splits;
  const int rt = id % a.row_tiles;
  id /= a.row_tiles;
  const int h = id % a.c.heads, seq = id / a.c.heads;
  const KvSeq s = kv_seq(a.b, seq, a.c.page_log2);
  const int rows = s.n * a.group, r0 = rt * (16 * NT);
  if (r0 >= rows) return;
  const int r1 = r0 + 16 * NT < rows ? r0 + 16 * NT : rows;  // one past the last
  Keys<kFewKeys> keys;
  keys.init(a, s, r0 / a.group, (r1 - 1) / a.group, split);

  const int lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  uint8_t* vt = lds + wave * (kFewKeys * 2 * D);

  // the lane's rows: query fragment, score scale, visible range
  x8 qf[NT][W], ql[LO ? NT : 1][W];
  float rs[NT];
  int hi_row[NT], lo_row[NT];
  const float sign = score_sign<MX>(a);
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int r = r0 + 16 * n + m;
    const bool has = r < r1;
    const int i = (has ? r : r1 - 1) / a.group, head = h * a.group + (has ? r : r1 - 1) - i * a.group;
    const uint16_t* q = a.q + (s.first + i) * a.q_token + head * a.q_head + g * (D / 4);
    float t[D / 4], mx = 0.0f;
#pragma unroll
    for (int k = 0; k < D / 64; ++k) {
      float x[16];
      load_q16(q + 16 * k, a.c.rht, a.c.signs, x);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        t[16 * k + e] = x[e] * sign;
        mx = fmaxf(mx, fabsf(x[e]));
      }
    }
    float down = 1.0f, up = 1.0f;
    if constexpr (!MX) row_power(max_over_g(mx), down, up);
    rs[n] = score_scale<MX>(a, up);
    const int64_t p = s.pos + i;
    hi_row[n] = (int)(p + 1 < 0 ? 0 : (p + 1 < s.kv ? p + 1 : s.kv));
    lo_row[n] = a.window > 0 && p + 1 > a.window ? (int)(p + 1 - a.window < s.kv ? p + 1 - a.window : s.kv) : 0;
#pragma unroll
    for (int j = 0; j < W; ++j) {
      w4 w, x;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float u = t[8 * j + 2 * e] * down, v = t[8 * j + 2 * e + 1] * down;
        w[e] = pack2<MX>(u, v);
        if constexpr (LO)
          x[e] = pack2<MX>(u - __uint_as_float(w[e] << 16), v - __uint_as_float(w[e] & 0xFFFF0000u));
      }
      qf[n][j] = as8<MX>(w);
      if constexpr (LO) ql[n][j] = as8<MX>(x);
    }
  }

  f32x4 o[NT][J], l[NT];
  float top[NT];  // the row's running maximum, shared by its four lanes
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    top[n] = -__builtin_inff();
    l[n] = f32x4{};
#pragma unroll
    for (int j = 0; j < J; ++j) o[n][j] = f32x4{};
  }
  const x8 ones = as8<MX>(w4{N::kOnes, N::kOnes, N::kOnes, N::kOnes});

  // rows of a transposing read: four tokens of the lane group, and the lane's
  // place in them
  const int tr_row = 4 * g + (m >> 2), tr_in = (m & 1) * 8, tr_piece = (m & 3) >> 1;
  // keys that every row of this workgroup sees
  const int64_t p0 = s.pos + r0 / a.group, p1 = s.pos + (r1 - 1) / a.group;
  const int all_hi = (int)(p0 + 1 < 0 ? 0 : (p0 + 1 < s.kv ? p0 + 1 : s.kv));
  const int64_t all_lo = a.window > 0 ? p1 + 1 - a.window : 0;

  FewTile<MX, D> cur, nxt;
  int u = keys.begin + wave;
  int page[2];
  if (u < keys.end) {
    const int t0 = keys.base(u);
    page[0] = page_of(a, seq, t0, keys.hi);
    page[1] = page_of(a, seq, t0 + 16, keys.hi);
    few_load<MX, D>(a, h, t0, keys.hi, page, cur);
    if (u + kFewWaves < keys.end) {
      const int t1 = keys.base(u + kFewWaves);
      page[0] = page_of(a, seq, t1, keys.hi);
      page[1] = page_of(a, seq, t1 + 16, keys.hi);
    }
  }
  for (; u < keys.end; u += kFewWaves) {
    const int t0 = keys.base(u);
    if (u + kFewWaves < keys.end) {
      few_load<MX, D>(a, h, keys.base(u + kFewWaves), keys.hi, page, nxt);
      if (u + 2 * kFewWaves < keys.end) {
        const int t2 = keys.base(u + 2 * kFewWaves);
        page[0] = page_of(a, seq, t2, keys.hi);
        page[1] = page_of(a, seq, t2 + 16, keys.hi);
      }
    }
    const bool inside = t0 + kFewKeys <= all_hi && t0 >= all_lo && cur.page[0] >= 0 && cur.page[1] >= 0;
    if (!inside) {
      // what no row sees may hold anything (it was never written, or its
      // page was given back): its codes and scales become zeros, so that
      // a probability of 0 meets no NaN
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int t = t0 + 16 * r + m;
        const bool ok = cur.page[r] >= 0 && t < keys.hi && (t >= keys.lo || t < a.sinks);
#pragma unroll
        for (int j = 0; j < W; ++j) cur.v[r][j] = ok ? cur.v[r][j] : 0u;
        cur.vs[r] = ok ? cur.vs[r] : 0u;
      }
    }
    // S^T = K q^T: registers i of tile r: key t0 + 16 r + 4 g + i
    f32x4 sc[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) sc[n][0] = sc[n][1] = f32x4{};
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int j = 0; j < W; ++j) {
        Scale<MX> k;
        block_scale(cur.ks[r], block_of_word<MX>(j), k);
        const x8 kf = as8<MX>(dequant8(cur.k[r][j], k));
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          sc[n][r] = N::mma(kf, qf[n][j], sc[n][r]);
          if constexpr (LO) sc[n][r] = N::mma(kf, ql[n][j], sc[n][r]);
        }
      }
    // V's rows to LDS
    wave_lds_fence();
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int j = 0; j < W; ++j) {
        Scale<MX> k;
        block_scale(cur.vs[r], block_of_word<MX>(j), k);
        *reinterpret_cast<w4*>(vt + few_at<D>(16 * r + m, g * W + j)) = dequant8(cur.v[r][j], k);
      }
    wave_lds_fence();

    x8 pf[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float v[8];
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i) v[4 * r + i] = sc[n][r][i];
      if (!inside) {
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int t = t0 + 16 * r + 4 * g + i;
            const bool seen = cur.page[r] >= 0 && t < hi_row[n] && (t >= lo_row[n] || t < a.sinks);
            v[4 * r + i] = seen ? v[4 * r + i] : -__builtin_inff();
          }
      }
      float mx = v[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) mx = fmaxf(mx, v[i]);
      mx *= rs[n];
      // The maximum only has to keep exp2 in range: it is raised when a
      // score passes it by 2^8 (FP16 holds probabilities to 2^16), which
      // after the first tiles is rare, and spares the exchange between the
      // row's lanes and the scaling of the output.
      if (__any(mx > top[n] + 8.0f)) {
        const float t = fmaxf(top[n], max_over_g(mx));
        const float f = t == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(top[n] - t);
        top[n] = t;
        l[n] *= f;
#pragma unroll
        for (int j = 0; j < J; ++j) o[n][j] *= f;
      }
      const float sub = top[n] == -__builtin_inff() ? 0.0f : top[n];
      w4 w;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = pack2<MX>(__builtin_amdgcn_exp2f(__builtin_fmaf(v[2 * i], rs[n], -sub)),
                         __builtin_amdgcn_exp2f(__builtin_fmaf(v[2 * i + 1], rs[n], -sub)));
      pf[n] = as8<MX>(w);
      l[n] = N::mma(ones, pf[n], l[n]);  // every register: the row's sum
    }
    // O^T += V^T P^T: contraction slots (g, i): key t0 + 4 g + i, then t0 +
    // 16 + 4 g + i - 4
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int at = few_at<D>(tr_row, 2 * j + tr_piece) + tr_in;
      const w2 x = read_tr16(vt + at), y = read_tr16(vt + at + 16 * 2 * D);
      const x8 vf = as8<MX>(w4{x.x, x.y, y.x, y.y});
#pragma unroll
      for (int n = 0; n < NT; ++n) o[n][j] = N::mma(vf, pf[n], o[n][j]);
    }
    cur = nxt;
  }

  // Join the four waves: every wave's rows and (m, l) through LDS, then a
  // thread per row and 16 columns.
  constexpr int P = D + 4;  // row pitch, floats
  float* om = reinterpret_cast<float*>(lds);
  float2* ml = reinterpret_cast<float2*>(lds + few_lds<D>() - 1024);
  for (int n = 0; n < NT; ++n) {
    __syncthreads();
#pragma unroll
    for (int k = 0; k < NT; ++k)
      if (k == n) {
#pragma unroll
        for (int j = 0; j < J; ++j)
          *reinterpret_cast<f32x4*>(om + (wave * 16 + m) * P + 16 * j + 4 * g) = o[k][j];
        if (g == 0) ml[wave * 16 + m] = make_float2(top[k], l[k][0]);
      }
    __syncthreads();
    const int row = threadIdx.x / J, d0 = (threadIdx.x % J) * 16;
    const int r = r0 + 16 * n + row;
    if (row >= 16 || r >= r1) continue;
    float t = -__builtin_inff();
#pragma unroll
    for (int w = 0; w < kFewWaves; ++w) t = fmaxf(t, ml[w * 16 + row].x);
    const float sub = t == -__builtin_inff() ? 0.0f : t;
    float sum = 0.0f, x[16] = {};
#pragma unroll
    for (int w = 0; w < kFewWaves; ++w) {
      const float2 e = ml[w * 16 + row];
      const float f = __builtin_amdgcn_exp2f(e.x - sub);
      sum += e.y * f;
#pragma unroll
      for (int k = 0; k < 16; ++k) x[k] += om[(w * 16 + row) * P + d0 + k] * f;
    }
    const int i = r / a.group, head = h * a.group + r - i * a.group;
    const int64_t token = s.first + i;
    if (a.splits == 1) {
      const float f = out_factor<MX>(a, sum);
#pragma unroll
      for (int k = 0; k < 16; ++k) x[k] *= f;
      if (a.c.rht) rht16_inverse(x, a.c.signs);
      store_out16(a, token, head, d0, x);
      if (a.lse && d0 == 0) a.lse[token * a.q_heads + head] = row_lse(t, sum);
    } else {
      const int64_t at = ((int64_t)split * a.b.tokens + token) * a.q_heads + head;
      if (d0 == 0) a.part_ml[at] = make_float2(t, sum);
      if (sum > 0.0f) {
        f32x4* p = reinterpret_cast<f32x4*>(a.part + at * D + d0);
#pragma unroll
        for (int k = 0; k < 4; ++k) p[k] = f32x4{x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]};
      }
    }
  }
}

// ============================================================ many new tokens
// 256 rows to a workgroup of eight waves, 32 rows to a wave, tiles of 64
// keys: the workgroup dequantizes a tile once into LDS (K and V, 16 bits),
// while the waves work on the tile before it; every wave takes its products
// from there.
constexpr int kManyThreads = 512, kManyRows = 256, kManyKeys = 64;

// LDS places of 16-byte piece p of row r.  K is read by 32 rows at one piece,
// V through the transposing read: four rows of two pairs of pieces to a half
// wave; both are written four rows and four pieces (every W-th) at a time.
template <int D>
__device__ __forceinline__ int many_k_at(int r, int p) {
  const int s = D == 64 ? (r >> 1) & 7 : r & 15;
  return r * (2 * D) + ((p ^ s) << 4);
}
template <int D>
__device__ __forceinline__ int many_v_at(int r, int p) {
  const int s = D == 64 ? 5 * ((r >> 1) & 1) : 5 * (r & 3);
  return r * (2 * D) + ((p ^ s) << 4);
}

// Elements of a 32-row output tile in a lane: register 4 b + i is column
// 8 b + 4 h + i (h: the lane's half), so a 16-group lies in eight registers
// of each of two lanes.  The inverse transform: columns 1, 2 and 8 apart are
// registers of the lane, 4 apart the other half's lane.
__device__ __forceinline__ void rotate_back32(f32x16& v, int half, uint32_t signs) {
#pragma unroll
  for (int gr = 0; gr < 2; ++gr) {
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = v[8 * gr + e];
#pragma unroll
    for (int st = 1; st < 8; st <<= 1) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (e & st) continue;
        const float p = x[e], q = x[e + st];
        x[e] = p + q;
        x[e + st] = p - q;
      }
      if (st == 2) {  // columns 4 apart come between those 2 and 8 apart
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float other = __shfl_xor(x[e], 32);
          x[e] = half ? other - x[e] : x[e] + other;
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int col = 8 * (e >> 2) + 4 * half + (e & 3);
      const float y = x[e] * 0.25f;
      v[8 * gr + e] = ((signs >> col) & 1u) ? -y : y;
    }
  }
}

template <bool MX, bool LO, int D>
__global__ __launch_bounds__(kManyThreads, 2) void kv_many_kernel(Args a) {
  typedef Num<MX> N;
  typedef typename N::x8 x8;
  constexpr int B = MX ? 32 : 16;
  constexpr int W = D / 32;      // words of codes of a thread's quarter row
  constexpr int QK = D / 16;     // S^T instructions of one 32-key tile
  constexpr int DT = D / 32;     // 32-column tiles of the output
  constexpr int kTile = kManyKeys * 2 * D;  // bytes of one tile of K or V
  __shared__ __align__(16) uint8_t lds[4 * kTile];  // two tiles of K and of V

  // row tiles with the most keys first: the last workgroups to run are short
  int id = blockIdx.x;
  const int h = id % a.c.heads;
  id /= a.c.heads;
  const int seq = id % a.b.batch;
  id /= a.b.batch;
  const int split = id % a.splits;
  const int rt = a.row_tiles - 1 - id / a.splits;
  const KvSeq s = kv_seq(a.b, seq, a.c.page_log2);
  const int rows = s.n * a.group, r0 = rt * kManyRows;
  if (r0 >= rows) return;
  const int r1 = r0 + kManyRows < rows ? r0 + kManyRows : rows;
  Keys<kManyKeys> keys;
  keys.init(a, s, r0 / a.group, (r1 - 1) / a.group, split);

  const int lane = threadIdx.x & 63, half = lane >> 5, qrow = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  // this wave's rows
  const int w0 = r0 + 32 * wave;
  const bool works = w0 < r1;
  const int w1 = w0 + 32 < r1 ? w0 + 32 : r1;
  const int r = works ? (w0 + qrow < r1 ? w0 + qrow : r1 - 1) : r0;
  const int qi = r / a.group, head = h * a.group + r - qi * a.group;

  x8 qf[QK], ql[LO ? QK : 1];
  float rs;
  {
    const uint16_t* q = a.q + (s.first + qi) * a.q_token + head * a.q_head;
    const float sign = score_sign<MX>(a);
    float mx = 0.0f, down = 1.0f, up = 1.0f;
    // a lane keeps columns 16 j + 8 half + 0..7; the rotation takes whole
    // 16-groups, which both halves compute
    if constexpr (!MX) {
#pragma unroll
      for (int j = 0; j < QK; ++j) {
        float x[16];
        load_q16(q + 16 * j, a.c.rht, a.c.signs, x);
#pragma unroll
        for (int e = 0; e < 16; ++e) mx = fmaxf(mx, fabsf(x[e]));
      }
      row_power(mx, down, up);
    }
    rs = score_scale<MX>(a, up);
#pragma unroll
    for (int j = 0; j < QK; ++j) {
      float x[16];
      load_q16(q + 16 * j, a.c.rht, a.c.signs, x);
      w4 w, y;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float u = (half ? x[8 + 2 * e] : x[2 * e]) * sign * down;
        const float v = (half ? x[9 + 2 * e] : x[2 * e + 1]) * sign * down;
        w[e] = pack2<MX>(u, v);
        if constexpr (LO)
          y[e] = pack2<MX>(u - __uint_as_float(w[e] << 16), v - __uint_as_float(w[e] & 0xFFFF0000u));
      }
      qf[j] = as8<MX>(w);
      if constexpr (LO) ql[j] = as8<MX>(y);
    }
  }
  const int64_t p = s.pos + qi;
  const int hi_row = (int)(p + 1 < 0 ? 0 : (p + 1 < s.kv ? p + 1 : s.kv));
  const int lo_row = a.window > 0 && p + 1 > a.window ? (int)(p + 1 - a.window < s.kv ? p + 1 - a.window : s.kv) : 0;
  // keys that every row of this wave sees, and keys that any row sees
  const int64_t p0 = s.pos + w0 / a.group, p1 = s.pos + (w1 - 1) / a.group;
  const int all_hi = (int)(p0 + 1 < 0 ? 0 : (p0 + 1 < s.kv ? p0 + 1 : s.kv));
  const int64_t all_lo = a.window > 0 ? p1 + 1 - a.window : 0;
  const int any_hi = works ? (int)(p1 + 1 < 0 ? 0 : (p1 + 1 < s.kv ? p1 + 1 : s.kv)) : 0;
  const int64_t any_lo = a.window > 0 ? p0 + 1 - a.window : 0;

  f32x16 o[DT];
#pragma unroll
  for (int j = 0; j < DT; ++j) o[j] = f32x16{};
  float top = -__builtin_inff(), l = 0.0f;  // l: this lane's keys only

  // Staging: threads 0..255 take K, 256..511 V: four threads to a row, a
  // quarter (D / 4 codes) each.
  const bool is_v = threadIdx.x >= 256;
  const int st_row = (threadIdx.x & 255) >> 2, st_seg = threadIdx.x & 3;
  const uint8_t* st_codes = is_v ? a.c.v_codes : a.c.k_codes;
  const uint8_t* st_scales = is_v ? a.c.v_scales : a.c.k_scales;
  uint32_t raw[W], raw_s = 0;
  auto fetch = [&](int t0) {
    const int t = t0 + st_row;
    int page = -1;
    if (t < keys.hi && (t >= keys.lo || t < a.sinks)) {
      page = a.b.page_table[seq * a.b.table_ld + (t >> a.c.page_log2)];
      if (page < 0 || page >= a.c.pages) page = -1;
    }
#pragma unroll
    for (int j = 0; j < W; ++j) raw[j] = 0;
    raw_s = 0;
    if (page >= 0) {  // the rest stays zero: a masked key meets no NaN
      const int64_t row = row_of(a, page, h, t);
      load_words(st_codes + row * (D / 2) + st_seg * (D / 8), raw);
      raw_s = load_scales<MX, D>(st_scales + row * (D / B), st_seg);
    }
  };
  auto stage = [&](int buf) {
    uint8_t* to = lds + buf * 2 * kTile + (is_v ? kTile : 0);
#pragma unroll
    for (int j = 0; j < W; ++j) {
      Scale<MX> k;
      block_scale(raw_s, block_of_word<MX>(j), k);
      const int pc = st_seg * W + j;
      *reinterpret_cast<w4*>(to + (is_v ? many_v_at<D>(st_row, pc) : many_k_at<D>(st_row, pc))) =
          dequant8(raw[j], k);
    }
  };
  // rows of a transposing read: lane group (half, column half), four tokens
  const int tr_lane = lane & 15, tr_dh = (lane >> 4) & 1;
  const int tr_row = 4 * half + (tr_lane >> 2);
  const int tr_piece = 2 * tr_dh + ((tr_lane & 3) >> 1), tr_in = (tr_lane & 1) * 8;

  // tiles without a page (the sequence gave it back) hold zeros, which are
  // not keys: their scores are masked by the page table in the masked path
  if (keys.begin < keys.end) {
    fetch(keys.base(keys.begin));
    stage(0);
  }
  for (int u = keys.begin; u < keys.end; ++u) {
    const int t0 = keys.base(u), buf = (u - keys.begin) & 1;
    if (u + 1 < keys.end) fetch(keys.base(u + 1));
    __syncthreads();
    const uint8_t* kt = lds + buf * 2 * kTile;
    const uint8_t* vt = kt + kTile;
    const bool skip = t0 >= any_hi || (t0 + kManyKeys <= any_lo && t0 >= a.sinks);
    if (!skip) {
      f32x16 sc[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        sc[c] = f32x16{};
#pragma unroll
        for (int j = 0; j < QK; ++j) {
          const x8 kf = as8<MX>(*reinterpret_cast<const w4*>(kt + many_k_at<D>(32 * c + qrow, 2 * j + half)));
          sc[c] = N::mma(kf, qf[j], sc[c]);
          if constexpr (LO) sc[c] = N::mma(kf, ql[j], sc[c]);
        }
      }
      bool pages = true;
      for (int t = t0; t < t0 + kManyKeys; t += 16)
        pages = pages && page_of(a, seq, t, keys.hi) >= 0;
      if (!(t0 + kManyKeys <= all_hi && t0 >= all_lo && pages)) {
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const int tb = t0 + 32 * c + 8 * b;  // eight keys of one page
            const bool has = page_of(a, seq, tb, keys.hi) >= 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int t = tb + 4 * half + i;
              const bool seen = has && t < hi_row && (t >= lo_row || t < a.sinks);
              sc[c][4 * b + i] = seen ? sc[c][4 * b + i] : -__builtin_inff();
            }
          }
      }
      float mx = sc[0][0];
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int i = 0; i < 16; ++i) mx = fmaxf(mx, sc[c][i]);
      mx *= rs;
      if (__any(mx > top + 8.0f)) {  // as above: the maximum is raised rarely
        const float t = fmaxf(top, fmaxf(mx, __shfl_xor(mx, 32)));
        const float f = t == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(top - t);
        top = t;
        l *= f;
#pragma unroll
        for (int j = 0; j < DT; ++j) o[j] *= f;
      }
      const float sub = top == -__builtin_inff() ? 0.0f : top;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {  // 16 keys: t0 + 32 c + 16 b + {4 half + i, 8 + 4 half + i}
          w4 w;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[c][8 * b + 2 * i], rs, -sub));
            const float y = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[c][8 * b + 2 * i + 1], rs, -sub));
            w[i] = pack2<MX>(x, y);
            if constexpr (MX) {
              l += __uint_as_float(w[i] << 16);
              l += __uint_as_float(w[i] & 0xFFFF0000u);
            } else {
              l += x;
              l += y;
            }
          }
          const x8 pf = as8<MX>(w);
          const int tr = 32 * c + 16 * b + tr_row;
#pragma unroll
          for (int j = 0; j < DT; ++j) {
            const w2 x = read_tr16(vt + many_v_at<D>(tr, 4 * j + tr_piece) + tr_in);
            const w2 y = read_tr16(vt + many_v_at<D>(tr + 8, 4 * j + tr_piece) + tr_in);
            o[j] = N::mma(as8<MX>(w4{x.x, x.y, y.x, y.y}), pf, o[j]);
          }
        }
      }
    }
    if (u + 1 < keys.end) stage(buf ^ 1);
  }

  if (!works || w0 + qrow >= r1) return;
  l += __shfl_xor(l, 32);  // both halves of a row are here or neither
  const int64_t token = s.first + qi;
  if (a.splits == 1) {
    const float f = out_factor<MX>(a, l);
    const int64_t at = token * a.out_token + head * a.out_head;
#pragma unroll
    for (int j = 0; j < DT; ++j) {
      o[j] *= f;
      if (a.c.rht) rotate_back32(o[j], half, a.c.signs);
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int d = 32 * j + 8 * b + 4 * half;
        if (a.out_f32)
          *reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + at + d) =
              f32x4{o[j][4 * b], o[j][4 * b + 1], o[j][4 * b + 2], o[j][4 * b + 3]};
        else
          *reinterpret_cast<w2*>(static_cast<uint16_t*>(a.out) + at + d) =
              w2{bf16_pair(o[j][4 * b], o[j][4 * b + 1]), bf16_pair(o[j][4 * b + 2], o[j][4 * b + 3])};
      }
    }
    if (a.lse && half == 0) a.lse[token * a.q_heads + head] = row_lse(top, l);
  } else {
    const int64_t at = ((int64_t)split * a.b.tokens + token) * a.q_heads + head;
    if (half == 0) a.part_ml[at] = make_float2(top, l);
    if (l > 0.0f) {
#pragma unroll
      for (int j = 0; j < DT; ++j)
#pragma unroll
        for (int b = 0; b < 4; ++b)
          *reinterpret_cast<f32x4*>(a.part + at * D + 32 * j + 8 * b + 4 * half) =
              f32x4{o[j][4 * b], o[j][4 * b + 1], o[j][4 * b + 2], o[j][4 * b + 3]};
    }
  }
}

// ================================================================== joining
// The splits of a row (of a sequence's new token and a query head: rows of
// no sequence are left alone): a workgroup per row, D / 4 threads to a split
// (four columns each), the splits dealt to its slots in order, the slots
// summed in order: the result does not depend on which workgroup finished
// first.
constexpr int kJoinThreads = 256;

template <bool MX, int D>
__global__ __launch_bounds__(kJoinThreads) void kv_join_kernel(Args a) {
  constexpr int C = D / 4, SL = kJoinThreads / C;
  __shared__ __align__(16) float sums[SL][D];
  __shared__ float slot_l[SL];
  const int i = blockIdx.x / a.q_heads, head = blockIdx.x - i * a.q_heads;
  const KvSeq s = kv_seq(a.b, blockIdx.y, a.c.page_log2);
  if (i >= s.n) return;
  const int64_t token = s.first + i;
  const int64_t row = token * a.q_heads + head, rows = a.b.tokens * a.q_heads;
  const int c = threadIdx.x % C, sl = threadIdx.x / C;
  const float2* ml = a.part_ml + row;
  float t = -__builtin_inff();
  for (int k = 0; k < a.splits; ++k) t = fmaxf(t, ml[k * rows].x);
  const float sub = t == -__builtin_inff() ? 0.0f : t;
  f32x4 x = {};
  float l = 0.0f;
  for (int k = sl; k < a.splits; k += SL) {
    const float2 e = ml[k * rows];
    if (!(e.y > 0.0f)) continue;
    const float f = __builtin_amdgcn_exp2f(e.x - sub);
    l += e.y * f;
    x += *reinterpret_cast<const f32x4*>(a.part + (k * rows + row) * D + 4 * c) * f;
  }
  *reinterpret_cast<f32x4*>(&sums[sl][4 * c]) = x;
  if (c == 0) slot_l[sl] = l;
  __syncthreads();
  if (threadIdx.x >= D / 16) return;
  const int d0 = threadIdx.x * 16;
  float y[16] = {};
  l = 0.0f;
#pragma unroll
  for (int n = 0; n < SL; ++n) {
    l += slot_l[n];
#pragma unroll
    for (int k = 0; k < 16; ++k) y[k] += sums[n][d0 + k];
  }
  const float f = out_factor<MX>(a, l);
#pragma unroll
  for (int k = 0; k < 16; ++k) y[k] *= f;
  if (a.c.rht) rht16_inverse(y, a.c.signs);
  store_out16(a, token, head, d0, y);
  if (a.lse && d0 == 0) a.lse[row] = row_lse(t, l);
}

// ===================================================================== host
template <bool MX, bool LO, int D>
hipError_t launch_d(const Args& a, const KvAttentionPlan& p, hipStream_t s) {
  const int64_t groups = (int64_t)a.b.batch * a.c.heads * p.row_tiles * p.splits;
  if (p.prompt) {
    kv_many_kernel<MX, LO, D><<<(unsigned)groups, kManyThreads, 0, s>>>(a);
  } else if (p.rows == 16) {
    kv_few_kernel<MX, LO, D, 1><<<(unsigned)groups, kFewThreads, 0, s>>>(a);
  } else {
    kv_few_kernel<MX, LO, D, 2><<<(unsigned)groups, kFewThreads, 0, s>>>(a);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  const dim3 grid((unsigned)a.b.max_q * (unsigned)a.q_heads, (unsigned)a.b.batch);
  kv_join_kernel<MX, D><<<grid, kJoinThreads, 0, s>>>(a);
  return hipGetLastError();
}

template <bool MX, bool LO>
hipError_t launch(const Args& a, const KvAttentionPlan& p, hipStream_t s) {
  switch (a.c.dim) {
    case 64: return launch_d<MX, LO, 64>(a, p, s);
    case 128: return launch_d<MX, LO, 128>(a, p, s);
    default: return launch_d<MX, LO, 256>(a, p, s);
  }
}

}  // namespace

KvAttentionPlan fp4_plan_kv_attention(const KvCacheArgs& c, const KvBatchArgs& b, int q_heads,
                                      int window, int sinks) {
  KvAttentionPlan p{};
  const int64_t rows = (int64_t)b.max_q * (q_heads / c.heads);
  p.prompt = rows > 64;
  p.rows = p.prompt ? kManyRows : (rows > 16 ? 32 : 16);
  p.row_tiles = (int)((rows + p.rows - 1) / p.rows);
  int64_t seen = b.max_kv;
  if (window > 0 && (int64_t)window + sinks + b.max_q < seen) seen = (int64_t)window + sinks + b.max_q;
  const int tile = p.prompt ? kManyKeys : kFewKeys;
  const int64_t tiles = (seen + tile - 1) / tile + 2;
  const int64_t groups = (int64_t)b.batch * c.heads * p.row_tiles;
  // enough workgroups to fill the chip, and tiles enough for each
  const int64_t want = p.prompt ? 512 : 1024;
  const int64_t least = p.prompt ? 8 : 8;  // tiles of a split at least
  int64_t n = groups > 0 ? want / groups : 1;
  if (n > tiles / least) n = tiles / least;
  if (n < 1) n = 1;
  if (n > 256) n = 256;
  p.splits = (int)n;
  if (n > 1) p.bytes = (size_t)(n * b.tokens * q_heads) * ((size_t)c.dim * 4 + 8);
  return p;
}

hipError_t fp4_launch_kv_attention(const KvAttentionLaunch& q, hipStream_t s) {
  const KvAttentionPlan p = fp4_plan_kv_attention(q.cache, q.batch, q.q_heads, q.window, q.sinks);
  Args a{};
  a.c = q.cache;
  a.b = q.batch;
  a.q = static_cast<const uint16_t*>(q.q);
  a.q_token = q.q_token;
  a.q_head = q.q_head;
  a.q_heads = q.q_heads;
  a.group = q.q_heads / q.cache.heads;
  a.scale = q.scale;
  a.window = q.window;
  a.sinks = q.sinks;
  a.out = q.out;
  a.out_f32 = q.out_dtype == 1;
  a.out_token = q.out_token;
  a.out_head = q.out_head;
  a.lse = q.lse;
  a.splits = p.splits;
  a.row_tiles = p.row_tiles;
  if (p.splits > 1) {
    const int64_t rows = (int64_t)p.splits * q.batch.tokens * q.q_heads;
    a.part = static_cast<float*>(q.workspace);
    a.part_ml = reinterpret_cast<float2*>(a.part + rows * q.cache.dim);
  }
  if (q.cache.format == kNVFP4) return launch<false, false>(a, p, s);
  return q.cache.rht ? launch<true, true>(a, p, s) : launch<true, false>(a, p, s);
}
