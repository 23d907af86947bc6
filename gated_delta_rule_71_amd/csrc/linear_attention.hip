// Linear attention with one decay per value head, over packed or batched sequences:
//
//     S_t = lambda S_{t-1} + k_t v_t^T,     o_t = scale q_t S_t,     lambda = exp(g_h)
//
// (S as stored, [K, V]).  A chunk of r tokens with local indices i, j = 0 .. r-1 and
// entering state S is, with w(n) = lambda^n and w(0) = 1 (also where lambda = 0),
//
//     o_i = s_intra sum_{j <= i} w(i-j) (q_i . k_j) v_j + s_inter w(i+off) q_i S
//     S'  = w(r) S + s_upd sum_j w(r-1-j+1-off) k_j v_j^T
//
// with s_intra = s_inter = scale, s_upd = 1, off = 1.  The gradients are the same
// operator in other roles.  With dS_t = scale q_t do_t^T + G_t, G_{t-1} = lambda dS_t
// and G_{T-1} the gradient of the final state,
//     dq_t = scale S_t do_t     q := do, k := v, v := k on the transposed state;
//     dk_t = dS_t v_t           time reversed, q := v, k := do, v := q, transposed state;
//     dv_t = dS_t^T k_t         time reversed, q := k, k := q, v := do,
// where the reversed roles carry G, which is already decayed when the next token reads
// it (off = 0), and put the scale into the state (s_intra = s_upd = scale, s_inter = 1).
//
// One workgroup runs one value head of a stretch of tokens through its chunks.  Each of its
// waves (four; eight for sums at borders with DV = 128) owns DV/4 or DV/8 value columns of the
// state, in accumulator registers for the whole stretch; only the 64 x 64 (float32: 32 x 32)
// decayed scores pass between waves.
//
// Windows.  Without a delta rule a stretch's effect on the state is a decay and a sum, so
// the packed tokens are cut at every `window` tokens, whatever the sequences, to fill the
// chip: (1) the sequence that crosses the end of a window (time reversed: its begin) is
// summed up there from zero, or from its initial state if it begins inside; (2) these sums
// are combined along the borders, H = lambda^window H + sum; (3) every window runs the
// pieces of sequences that it holds, from their initial states or the state at its
// border.  Only (1) and (3) read tokens, k and v twice and the rest once.
//
// Bounds (36112 packed tokens, 32 heads of 128 x 128 on 16 q/k heads, bf16: 0.92 GB that a
// call must move, 182 us at a large copy's 5.07 TB/s; a call takes 422 us).  Medians of 200
// traced calls: (3) 299 us, 3.1 TB/s, with the matrix cores 29 percent and LDS 30 percent
// busy.  A chunk is a chain of loads, LDS, products and barriers that two workgroups per
// compute unit (registers, LDS) only partly hide.  (1) takes 121 us for k and v, (2) 7 us.
// One long prompt (16383 tokens, 16 heads, 129 us): 81, 42 and 12 us.  Gradients (4 x 4096
// tokens, 16 heads, 268 us): 199 us for the three roles, which share operands in L2, 64 and
// 8 us.  These have memories of one to 256 tokens; where all heads keep thousands, every token
// is in reach of a border: 451, 138 and 275 us.  Small calls pay the start of a workgroup (6 of
// 14 us for 97 tokens: cold code, tables, states).

#include "common.hpp"
#include "gdr_internal.hpp"

namespace gdr {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// ---- operands -----------------------------------------------------------------------
// A 16x16 product over a 32-deep slice: lane l = 16 g + c supplies row (A) or column (B)
// c at the contraction indices 8 g + e, e = 0..7, and receives D[4 g + i][c], i = 0..3.
//
// Parts.  A float32 value that meets a bf16 matrix-core operand is written as a sum of bf16
// values, each the rounding of what the ones before left (by at most 2^-8): two parts leave
// 2^-16 of the value, three 2^-24.
//  * The state and the scores take two where they meet q and v.  A result that is rounded to
//    bf16 then errs like the rounded exact one, and a float32 result keeps 16 bits of a term.
//    With one part the outputs err by 0.0023 of their norm in place of 0.0017, float32 ones
//    by as much (packed prefill 366 us in place of 422, gradients 251 in place of 269).
//  * The decayed values, which build the float32 states, take three where they are a part
//    of a state that is handed out, so that it is as exact as a float32 sum: all tokens whose
//    weight in it is not zero, as far ones can be all that it has (large at a prompt's start,
//    zeros behind; with two parts throughout 375 and 255 us).  Two where the state only
//    meets q.
// Matrix-core products a 64-token chunk at K = V = 128: 776 and 648 of 16x16x32; at a border
// 384 and 256.

template <typename T> struct Op;

template <> struct Op<uint16_t> {
  using elem = uint16_t;
  static constexpr int kChunk = 64;
  static constexpr int kStateParts = 2, kScoreParts = 2, kValueParts = 3;
  using frag = bf16x8;
  static __device__ __forceinline__ f32x4 mma(const frag &a, const frag &b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  // row `row` of a row-major LDS matrix at contraction indices k0 + 8 g + e
  static __device__ __forceinline__ frag rows(const elem *base, int ld, int row, int k0, int g) {
    return *reinterpret_cast<const frag *>(base + row * ld + k0 + 8 * g);
  }
  // column index c of a row-major LDS matrix at rows (contraction) r0 + 8 g + e, where
  // column index 4 m + n names column col0 + step m + n: transposed reads, for which lane
  // s of a 16-lane group names the 8 bytes at row s / 4, column group s % 4
  static __device__ __forceinline__ frag cols(const elem *base, int ld, int r0, int col0, int step,
                                              int lane) {
    const int g = lane >> 4, s = lane & 15;
    const elem *p = base + (r0 + 8 * g + (s >> 2)) * ld + col0 + step * (s & 3);
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) s16x4 *)(p));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) s16x4 *)(p + 4 * ld));
    return __builtin_bit_cast(frag, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  }
  static __device__ __forceinline__ void expand(const frag &f, float (&x)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = static_cast<float>(f[e]);
  }
  // One pair's next part, and what it leaves: hi = bf16(x), x - hi.  The subtraction is a
  // two-term bf16 dot product of the pair as it was rounded with (-1, 0) or (0, -1), exact,
  // which saves taking the halves apart.  The constants are kept from the compiler, which
  // would make them inline constants that select the wrong half.
  static __device__ __forceinline__ bf16x2 part(float &x0, float &x1, bool more) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const bf16x2 hi = __builtin_convertvector((f32x2{x0, x1}), bf16x2);
    if (more) {
      uint32_t lo_one = 0x0000bf80u, hi_one = 0xbf800000u;
      asm("" : "+s"(lo_one), "+s"(hi_one));
      x0 = __builtin_amdgcn_fdot2_f32_bf16(hi, __builtin_bit_cast(bf16x2, lo_one), x0, false);
      x1 = __builtin_amdgcn_fdot2_f32_bf16(hi, __builtin_bit_cast(bf16x2, hi_one), x1, false);
    }
    return hi;
  }
  template <int N>
  static __device__ __forceinline__ void parts(const float (&x)[8], frag (&f)[N]) {
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      float x0 = x[e], x1 = x[e + 1];
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const bf16x2 h = part(x0, x1, n + 1 < N);
        f[n][e] = h[0];
        f[n][e + 1] = h[1];
      }
    }
  }
  // four consecutive scores, a part to each matrix
  static __device__ __forceinline__ void store4(elem *p, int stride, float (&x)[4]) {
#pragma unroll
    for (int n = 0; n < kScoreParts; ++n) {
      const bool more = n + 1 < kScoreParts;
      const bf16x2 a = part(x[0], x[1], more), b = part(x[2], x[3], more);
      *reinterpret_cast<uint2 *>(p + n * stride) =
          make_uint2(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b));
    }
  }
};

template <> struct Op<float> {
  using elem = float;
  static constexpr int kChunk = 32;
  static constexpr int kStateParts = 1, kScoreParts = 1, kValueParts = 1;
  struct frag { float v[8]; };
  static __device__ __forceinline__ f32x4 mma(const frag &a, const frag &b, f32x4 c) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[e], b.v[e], c, 0, 0, 0);
    return c;
  }
  static __device__ __forceinline__ frag rows(const elem *base, int ld, int row, int k0, int g) {
    frag f;
    load8(base + row * ld + k0 + 8 * g, f.v);
    return f;
  }
  static __device__ __forceinline__ frag cols(const elem *base, int ld, int r0, int col0, int step,
                                              int lane) {
    const int g = lane >> 4, s = lane & 15;
    const elem *p = base + (r0 + 8 * g) * ld + col0 + step * (s >> 2) + (s & 3);
    frag f;
#pragma unroll
    for (int e = 0; e < 8; ++e) f.v[e] = p[e * ld];
    return f;
  }
  static __device__ __forceinline__ void expand(const frag &f, float (&x)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = f.v[e];
  }
  template <int N>
  static __device__ __forceinline__ void parts(const float (&x)[8], frag (&f)[N]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[0].v[e] = x[e];
  }
  static __device__ __forceinline__ void store4(elem *p, int, float (&x)[4]) {
    *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
  }
};

// lambda^n from the log-decay g: 1 at n = 0 whatever g; n g in two floats, so that the
// power's error stays an ulp for far tokens.
__device__ __forceinline__ float decay_power(float g, int n) {
  if (n == 0) return 1.0f;
  const float x = static_cast<float>(n) * g;
  const float e = expf(x);
  if (!(g < 0.0f) || x < -1.0e30f) return e;
  return fmaf(e, fmaf(static_cast<float>(n), g, -x), e);
}

// Tokens after which a head's weight is zero: exp(-104) is below half of float32's least
// number.  What lies farther back adds nothing.
__device__ __forceinline__ long decay_reach(float g) {
  return g < 0.0f ? static_cast<long>(fminf(ceilf(104.0f / -g), 1.0e9f)) : 1L << 40;
}

// Four lanes' four elements, transposed: lane 4 q + j gets element j of lanes 4 q .. 4 q + 3.
__device__ __forceinline__ f32x4 transpose4(f32x4 x, int lane) {
  auto swap = [](float v, auto ctrl) {
    return __int_as_float(
        __builtin_amdgcn_update_dpp(0, __float_as_int(v), decltype(ctrl)::value, 0xf, 0xf, true));
  };
  using one = std::integral_constant<int, 0xB1>;   // quad_perm 1, 0, 3, 2
  using two = std::integral_constant<int, 0x4E>;   // quad_perm 2, 3, 0, 1
  const bool odd = lane & 1, high = lane & 2;
  const float a = swap(odd ? x[0] : x[1], one()), b = swap(odd ? x[2] : x[3], one());
  x = odd ? f32x4{a, x[1], b, x[3]} : f32x4{x[0], a, x[2], b};
  const float u = swap(high ? x[0] : x[2], two()), v = swap(high ? x[1] : x[3], two());
  return high ? f32x4{u, v, x[2], x[3]} : f32x4{x[0], x[1], u, v};
}

// N consecutive outputs (the hardware's rounding to nearest even)
template <int N>
__device__ __forceinline__ void store_out(uint16_t *p, const float (&x)[N]) {
  typedef __bf16 bf16xN __attribute__((ext_vector_type(N)));
  bf16xN y;
#pragma unroll
  for (int i = 0; i < N; ++i) y[i] = static_cast<__bf16>(x[i]);
  *reinterpret_cast<bf16xN *>(p) = y;
}
template <int N>
__device__ __forceinline__ void store_out(float *p, const float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4)
    *reinterpret_cast<float4 *>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
}

// Workgroups per head and role: windows or sequences; borders, and again for the copies of
// the initial states of sequences that cross them.
__host__ __device__ inline int linear_places(const LinearParams &p, bool output) {
  if (output) return p.window ? p.windows : p.num_seqs;
  return (p.windows - 1) * (p.role[0].saved ? 2 : 1);
}

// 16-column tiles of a wave where V = 128: two share their reads of q and k where outputs
// are formed; one each, on twice the waves, at the borders.
constexpr int cols(bool output) { return output ? 2 : 1; }
constexpr int threads(int dv, bool output) { return dv == 128 ? 512 / cols(output) : 256; }

template <typename T, int DQ, int DV, bool OUTPUT> struct Lds {
  static constexpr int C = Op<T>::kChunk;
  // Rows padded by 16 bytes for 16-byte reads of 16 rows (7.1 cycles a wave instruction, 32
  // without padding) and transposed reads of adjacent columns; by 64 where the transposed
  // reads take every other group of four columns (4.4 cycles; 8.0 with 16 bytes).
  static constexpr int kPad = 16 / sizeof(T), kPadTr = sizeof(T) == 2 ? 32 : kPad;
  static constexpr int ldq = DQ + kPad, ldk = DQ + kPadTr, ldv = DV + (DV == 128 && cols(OUTPUT) == 2 ? kPadTr : kPad), lds = C + kPad;
  T q[OUTPUT ? C * ldq : 8];   // the sums at the borders use neither q nor scores
  T k[C * ldk];
  T v[C * ldv];
  alignas(16) T score[Op<T>::kScoreParts][OUTPUT ? C * lds : 8];
  float pw[C + 1];
  // s_intra times the weight of key 4 g + e behind token c, the tiles 16 * [i] tokens apart
  alignas(16) float gap[OUTPUT ? C / 16 : 1][64][4];
  int mark;           // a value of the chunk is not finite
  float upd[2 * C];   // the update's weights, those of r tokens from upd[C - r] on
};

// Eight consecutive input elements in registers, as whole 16-byte vectors.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
template <typename T> struct Vec8 {
  static constexpr int N = 8 * sizeof(T) / 16;
  u32x4 u[N];
  __device__ __forceinline__ void load(const char *p) {
#pragma unroll
    for (int n = 0; n < N; ++n) u[n] = reinterpret_cast<const u32x4 *>(p)[n];
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int n = 0; n < N; ++n) u[n] = u32x4{0, 0, 0, 0};
  }
  __device__ __forceinline__ void store(T *p) const {
#pragma unroll
    for (int n = 0; n < N; ++n) reinterpret_cast<u32x4 *>(p)[n] = u[n];
  }
  // Top bits set where an element is not finite: exponents of ones leave a zero that the
  // subtraction of one turns negative (a borrow into the next half only follows a hit).
  __device__ __forceinline__ uint32_t not_finite() const {
    const uint32_t m = sizeof(T) == 2 ? 0x7f807f80u : 0x7f800000u;
    const uint32_t one = sizeof(T) == 2 ? 0x00010001u : 1u;
    uint32_t mark = 0;
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int w = 0; w < 4; ++w) mark |= (~u[n][w] & m) - one;
    return mark & (sizeof(T) == 2 ? 0x80008000u : 0x80000000u);
  }
};

// Rows [0, r) of a chunk's operand (row i is token i from the chunk's lowest token on, or
// token r - 1 - i in reverse), zeros behind them, from memory to registers and on to LDS.
// All loads of a chunk are in flight before the first is waited for; rows behind the last
// one read the lowest token and drop it, without a branch between the loads.
template <typename T, int D, int NT> struct Tile {
  static constexpr int kSegs = Op<T>::kChunk * (D / 8), kRows = NT / (D / 8);
  static constexpr int N = (kSegs + NT - 1) / NT;   // below one for the smallest tiles
  Vec8<T> s[N];
  // low: the chunk's lowest token (uniform); step: bytes from token to token
  __device__ __forceinline__ void load(const char *low, uint32_t step, int r, bool reverse) {
    const int row = threadIdx.x / (D / 8);
    const uint32_t col = 8 * (threadIdx.x % (D / 8)) * sizeof(T);
#pragma unroll
    for (int m = 0; m < N; ++m) {
      const int i = row + m * kRows;
      s[m].load(low + (i < r ? (reverse ? r - 1 - i : i) * step + col : col));
    }
  }
  // to LDS; whether an element is not finite
  __device__ __forceinline__ uint32_t store(T *dst, int ld, int r) {
    const int row = threadIdx.x / (D / 8), col = 8 * (threadIdx.x % (D / 8));
    uint32_t mark = 0;
    if (r < Op<T>::kChunk) {
#pragma unroll
      for (int m = 0; m < N; ++m)
        if (row + m * kRows >= r) s[m].zero();
    }
#pragma unroll
    for (int m = 0; m < N; ++m) {
      if (kSegs < NT && threadIdx.x >= kSegs) break;
      mark |= s[m].not_finite();
      s[m].store(dst + (row + m * kRows) * ld + col);
    }
    return mark;
  }
};

// First tokens and states of the sequences.  Up to 63 of them sit in the lanes of one
// register each, so that a workgroup starts after one trip to memory instead of four.
struct Sequences {
  const LinearParams &p;
  const int lane;
  const bool held;
  int cu = 0, slots = 0;
  __device__ __forceinline__ Sequences(const LinearParams &params, int l)
      : p(params), lane(l), held(params.num_seqs < 64) {
    if (!held) return;
    if (p.cu_seqlens) cu = p.cu_seqlens[min(lane, p.num_seqs)];
    if (p.state_indices) slots = p.state_indices[min(lane, p.num_seqs - 1)];
  }
  __device__ __forceinline__ long begin(int n) const {
    if (!p.cu_seqlens) return static_cast<long>(n) * p.seqlen;
    return held ? __builtin_amdgcn_readlane(cu, n) : p.cu_seqlens[n];
  }
  __device__ __forceinline__ int slot(int n) const {
    if (!p.state_indices) return n;
    return held ? __builtin_amdgcn_readlane(slots, n) : p.state_indices[n];
  }
  // the first sequence that ends at `at` or behind it (the whole wave calls)
  __device__ __forceinline__ int ending_at(long at) const {
    if (!p.cu_seqlens)
      return static_cast<int>(max((at + p.seqlen - 1) / p.seqlen - 1, 0L));
    if (held) return __popcll(__ballot(lane >= 1 && lane <= p.num_seqs && cu < at));
    // 64 places looked up at a time: the sequences before n end before `at`, number `end`
    // (if there is one) does not
    int n = 0;
    for (int end = p.num_seqs; n < end;) {
      const int step = (end - n + 63) / 64, m = n + (lane + 1) * step - 1;
      const int before = __popcll(__ballot(m < end && p.cu_seqlens[m + 1] < at));
      n = min(n + before * step, end);
      end = min(n + step - 1, end);
    }
    return n;
  }
};

// OUTPUT: the outputs and final states of a window's (or sequence's) pieces; else the sum
// at the window's border.
template <typename T, int DQ, int DV, bool OUTPUT>
__global__ void __launch_bounds__(threads(DV, OUTPUT), OUTPUT ? 2 : 4) linear_attention_kernel(const LinearParams p) {
  using O = Op<T>;
  using L = Lds<T, DQ, DV, OUTPUT>;
  constexpr int C = O::kChunk;
  constexpr int KT = DQ / 16;       // state row tiles
  constexpr int NT = threads(DV, OUTPUT);
  constexpr int CT = 4 * DV / NT;   // column tiles of a wave
  constexpr int WAVES = NT / 64;
  constexpr int IT = C / 16;        // token tiles
  constexpr int JS = C / 32;        // token slices
  constexpr int KS = DQ / 32;       // key slices
  constexpr int TILES = IT * (IT + 1) / 2, SLOTS = (TILES + WAVES - 1) / WAVES;   // of scores
  __shared__ L lds;

  // the roles and grouped heads of one place share operands: on one XCD, side by side
  const uint32_t members = (p.roles * p.group) << p.halves, step = blockIdx.x >> 3;
  const uint32_t set = step / members * 8 + (blockIdx.x & 7), Hk = p.Hk, hk = set % Hk;
  const uint32_t part = step % members, member = part >> p.halves;
  const int V = DV << p.halves, vcol0 = part & p.halves ? DV : 0;   // value columns, first one
  int place = set / Hk;
  if (place >= linear_places(p, OUTPUT)) return;
  const uint32_t role = member / static_cast<uint32_t>(p.group);
  const int h = hk * p.group + member - role * p.group;
  const LinearRole &R = p.role[role];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);   // uniform
  const int g = lane >> 4, c = lane & 15;
  const Sequences seqs(p, lane);
  const float gh = p.g[h];

  // Row m of state tile kt is key row 32 (kt / 2) + 8 (m / 4) + 4 (kt % 2) + m % 4: a
  // lane's accumulators of two state tiles are then the eight contraction indices of an
  // operand.  Index n of column tile ct is value column 4 CT (n / 4) + 4 ct + n % 4 of the
  // wave: its tiles' accumulators are consecutive columns.
  const int col0 = 16 * CT * wave;
  f32x4 S[KT][CT];
  const size_t state_size = static_cast<size_t>(DQ) * V;
  // States in memory, 16 bytes per lane: a lane's four elements are consecutive where rows
  // are (state_rs = 1); else four lanes swap theirs, so that each has a row's columns.
  const bool by_rows = R.state_rs != 1;
  const uint32_t state_lane =
      by_rows ? (8 * g + (c & 3)) * R.state_rs + vcol0 + col0 + 4 * CT * (c >> 2)
              : 8 * g + (vcol0 + col0 + 4 * CT * (c >> 2) + (c & 3)) * R.state_cs;
  auto state_tile = [&](int kt, int ct) {
    return (32 * (kt / 2) + 4 * (kt % 2)) * R.state_rs + 4 * ct * R.state_cs;
  };
  auto load_state = [&](const float *src, size_t index) {
    if (src) {
      src += (index * p.H + h) * state_size;
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
          S[kt][ct] = *reinterpret_cast<const f32x4 *>(src + state_tile(kt, ct) + state_lane);
      if (by_rows)
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
          for (int ct = 0; ct < CT; ++ct) S[kt][ct] = transpose4(S[kt][ct], lane);
    } else {
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) S[kt][ct] = zero4();
    }
  };
  auto store_state = [&](float *dst, size_t index) {
    dst += (index * p.H + h) * state_size;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
        *reinterpret_cast<f32x4 *>(dst + state_tile(kt, ct) + state_lane) =
            by_rows ? transpose4(S[kt][ct], lane) : S[kt][ct];
  };

  int ti[SLOTS], tj[SLOTS];   // the wave's score tiles
#pragma unroll
  for (int m = 0; m < SLOTS; ++m) {
    ti[m] = 0;
    tj[m] = m * WAVES + wave;
    while (tj[m] > ti[m]) tj[m] -= ++ti[m];
  }

  const long reach = decay_reach(gh);
  const int off = R.reverse ? 0 : 1;
  if (threadIdx.x == 0) lds.mark = 0;
  for (int i = threadIdx.x; i <= C; i += NT) lds.pw[i] = decay_power(gh, i);
  __syncthreads();
  if constexpr (OUTPUT)
    for (int i = threadIdx.x; i < C / 16 * 256; i += NT) {
      const int l = (i >> 2) & 63, n = 16 * (i >> 8) + (l & 15) - 4 * (l >> 4) - (i & 3);
      lds.gap[0][0][i] = n >= 0 ? R.s_intra * lds.pw[max(n, 0)] : 0.0f;
    }
  for (int i = threadIdx.x; i < 2 * C; i += NT)
    lds.upd[i] = i < C ? R.s_upd * lds.pw[max(C - i - off, 0)] : 0.0f;
  // score tiles above the diagonal stay zero
  if constexpr (OUTPUT)
    for (int i = threadIdx.x; i < static_cast<int>(sizeof(lds.score)) / 16; i += NT)
      reinterpret_cast<u32x4 *>(lds.score)[i] = u32x4{0, 0, 0, 0};

  // heads and head of an operand: the value heads, or the q/k heads (div: of `group`)
  auto heads = [&](int div) { return static_cast<uint32_t>(div == 1 ? p.H : p.Hk); };
  auto head = [&](int div) { return static_cast<uint32_t>(div == 1 ? h : hk); };
  const uint32_t sq = heads(R.div_q) * DQ * sizeof(T), sk = heads(R.div_k) * DQ * sizeof(T),
                 sv = heads(R.div_v) * V * sizeof(T);   // bytes from token to token
  const uint32_t so = p.H * V * (R.out_f32 ? 4 : 2);
  const char *q = static_cast<const char *>(R.q) + head(R.div_q) * DQ * sizeof(T);
  const char *k = static_cast<const char *>(R.k) + head(R.div_k) * DQ * sizeof(T);
  const char *v = static_cast<const char *>(R.v) + (head(R.div_v) * V + vcol0) * sizeof(T);
  char *out = static_cast<char *>(R.out) + (h * V + vcol0) * (R.out_f32 ? 4 : 2);

  // The place's tokens [w0, w1), its first sequence, and whether it is the last place that
  // holds tokens (which then has the empty sequences at the end, too).
  const long total = seqs.begin(p.num_seqs);
  long w0 = 0, w1 = total;
  int n = place;
  bool last = false;
  if constexpr (OUTPUT) {
    if (p.window) {
      w0 = static_cast<long>(place) * p.window;
      if (w0 >= total && place > 0) return;
      w1 = min(w0 + p.window, total);
      last = w1 == total;
      n = seqs.ending_at(w0);
    }
  } else {
    // the sequence that holds the tokens on both sides of the border, and the window on the
    // side that its steps come from
    const bool copy = place >= p.windows - 1;
    if (copy) place -= p.windows - 1;
    const long border = static_cast<long>(place + 1) * p.window;
    w0 = border - (R.reverse ? 0 : p.window);
    w1 = min(w0 + p.window, total);
    n = seqs.ending_at(border + 1);
    const bool crosses = n < p.num_seqs && seqs.begin(n) < border;
    if (copy) {   // the initial state, for the window that the sequence begins in
      if (!crosses || seqs.begin(n) < w0 || !R.initial_state) return;
      const long from = static_cast<long>(max(seqs.slot(n), 0)) * p.H + h;
      const long to = static_cast<long>(place) * p.H + h;
      const f32x4 *src = reinterpret_cast<const f32x4 *>(R.initial_state + from * state_size + DQ * vcol0);
      f32x4 *dst = reinterpret_cast<f32x4 *>(R.saved + to * state_size + DQ * vcol0);
#pragma unroll
      for (int i = 0; i < DQ * DV / 4 / NT; ++i) dst[threadIdx.x + i * NT] = src[threadIdx.x + i * NT];
      return;
    }
    if (h == 0 && threadIdx.x == 0) {
      const bool more = crosses && (R.reverse ? seqs.begin(n + 1) > w1 : seqs.begin(n) < w0);
      R.crossing[place] = more ? 2 : crosses;
    }
    if (!crosses) return;
  }

  // every sequence with tokens in the window and the empty ones at its tokens; or the one
  // sequence of the place, or that crosses
  for (; n < p.num_seqs; ++n) {
    const long t0 = seqs.begin(n), t1 = seqs.begin(n + 1);
    long a = t0, b = t1;
    if (!OUTPUT || p.window) {
      if (OUTPUT && t0 >= w1 && !last) break;
      if (OUTPUT && t1 == w0 && t0 < w0) continue;   // ended where the window begins
      a = max(t0, w0);
      b = min(t1, w1);
    }
    if constexpr (!OUTPUT) {
      // only the tokens that the border is in reach of
      if (R.reverse) b = min(b, a + reach);
      else a = max(a, b - reach);
    }
    const int slot = seqs.slot(n);
    // a is t0 (reversed: b is t1) where the piece has the sequence's first step
    const bool first = R.reverse ? b == t1 : a == t0, done_here = R.reverse ? a == t0 : b == t1;
    // A chunk's operands are loaded while the chunk before it is computed.  `low` is the
    // lowest token of the `r` tokens at hand.
    long left = b - a;
    int r = static_cast<int>(min(static_cast<long>(C), left));
    long low = R.reverse ? b - r : a;
    Tile<T, DQ, NT> tq, tk;
    Tile<T, DV, NT> tv;
    auto load_tiles = [&](long at, int rows) {
      if constexpr (OUTPUT) tq.load(q + at * sq, sq, rows, R.reverse);
      tk.load(k + at * sk, sk, rows, R.reverse);
      tv.load(v + at * sv, sv, rows, R.reverse);
    };
    auto store_tiles = [&](int rows) {
      if constexpr (OUTPUT) tq.store(lds.q, L::ldq, rows);
      tk.store(lds.k, L::ldk, rows);
      return tv.store(lds.v, L::ldv, rows);
    };
    if (left > 0) load_tiles(low, r);
    if constexpr (OUTPUT) {
      if (!first)
        load_state(R.carried, place - 1 + R.reverse);
      else if (!done_here && R.saved)   // its slot may already hold the final state
        load_state(R.initial_state ? R.saved : nullptr, place);
      else
        load_state(R.initial_state, slot < 0 ? 0 : slot);
    } else {
      load_state(first ? R.initial_state : nullptr, slot < 0 ? 0 : slot);
    }
    for (int next; left > 0; r = next) {
      __syncthreads();
      const uint32_t bad = store_tiles(r);
      if (OUTPUT && bad) lds.mark = 1;
      __syncthreads();
      const long base = low, after = left - r;
      const bool exact = R.exact_state && (R.reverse ? low - t0 : t1 - low - r) < reach;
      next = static_cast<int>(min(static_cast<long>(C), after));
      if (after > 0) load_tiles(R.reverse ? low - next : low + r, next);

      // Decayed scores, tiles on and below the diagonal: D[j][i], four keys j per lane.  The
      // wave's tiles run side by side, as each one's products wait for one another.
      if constexpr (OUTPUT) {
        f32x4 d[SLOTS];
#pragma unroll
        for (int m = 0; m < SLOTS; ++m) d[m] = zero4();
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int m = 0; m < SLOTS; ++m)
            if (m * WAVES + wave < TILES)
              d[m] = O::mma(O::rows(lds.k, L::ldk, 16 * tj[m] + c, 32 * s, g),
                            O::rows(lds.q, L::ldq, 16 * ti[m] + c, 32 * s, g), d[m]);
        // A value that is not finite, times the zero scores of the tokens before it, would
        // make those tokens' outputs NaN: up to such a token the chunks have one token.  Each
        // of them is tried whole again first, which such inputs may cost: one NaN in the middle
        // of 16383 tokens makes the call 507 us in place of 129, NaN throughout 4.6 ms.
        if (lds.mark) {
          __syncthreads();
          lds.mark = 0;
          if (r > 1) {
            if (R.reverse) low += r - 1;
            next = 1;
            load_tiles(low, next);
            continue;
          }
        }
#pragma unroll
        for (int m = 0; m < SLOTS; ++m) {
          if (m * WAVES + wave >= TILES) break;
          const f32x4 w = *reinterpret_cast<const f32x4 *>(lds.gap[ti[m] - tj[m]][lane]);
          float x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)   // masked, not weighted: a key behind may not be finite
            x[e] = ti[m] > tj[m] || c >= 4 * g + e ? d[m][e] * w[e] : 0.0f;
          O::store4(lds.score[0] + (16 * ti[m] + c) * L::lds + 16 * tj[m] + 4 * g, C * L::lds, x);
        }
      }

      low = R.reverse ? low - next : low + r;
      left = after;

      f32x4 acc[CT][IT];
      typename O::frag vf[JS][CT];
#pragma unroll
      for (int js = 0; js < JS; ++js)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
          vf[js][ct] = O::cols(lds.v, L::ldv, 32 * js, col0 + 4 * ct, 4 * CT, lane);
      if constexpr (OUTPUT) {
        // outputs: acc[ct][it] holds value columns (rows) of tokens 16 it + c (columns)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
          for (int it = 0; it < IT; ++it) acc[ct][it] = zero4();
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          typename O::frag sf[CT][O::kStateParts];
#pragma unroll
          for (int ct = 0; ct < CT; ++ct) {
            float x[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              x[e] = S[2 * s][ct][e];
              x[4 + e] = S[2 * s + 1][ct][e];
            }
            O::parts(x, sf[ct]);
          }
          // products of one accumulator apart from each other, here and below: a dependent
          // one would wait out its predecessor's latency
#pragma unroll
          for (int it = 0; it < IT; ++it) {
            const typename O::frag qf = O::rows(lds.q, L::ldq, 16 * it + c, 32 * s, g);
#pragma unroll
            for (int n2 = 0; n2 < O::kStateParts; ++n2)
#pragma unroll
              for (int ct = 0; ct < CT; ++ct) acc[ct][it] = O::mma(sf[ct][n2], qf, acc[ct][it]);
          }
        }
        __syncthreads();   // the scores of the other waves
#pragma unroll
        for (int it = 0; it < IT; ++it) {
          const float w = R.s_inter * lds.pw[16 * it + c + off];
#pragma unroll
          for (int ct = 0; ct < CT; ++ct) acc[ct][it] *= w;
        }
#pragma unroll
        for (int js = 0; js < JS; ++js)
          for (int n2 = 0; n2 < O::kScoreParts; ++n2)
#pragma unroll
            for (int it = 2 * js; it < IT; ++it) {
              const typename O::frag af = O::rows(lds.score[n2], L::lds, 16 * it + c, 32 * js, g);
#pragma unroll
              for (int ct = 0; ct < CT; ++ct) acc[ct][it] = O::mma(vf[js][ct], af, acc[ct][it]);
            }
      }

      if constexpr (OUTPUT) {
        char *rows = out + base * so;
        auto put = [&](int it) {
          float y[4 * CT];
#pragma unroll
          for (int ct = 0; ct < CT; ++ct)
#pragma unroll
            for (int i = 0; i < 4; ++i) y[4 * ct + i] = acc[ct][it][i];
          const uint32_t token = R.reverse ? r - 1 - (16 * it + c) : 16 * it + c;
          const int col = col0 + 4 * CT * g;
          if (R.out_f32)
            store_out<4 * CT>(reinterpret_cast<float *>(rows + (token * so + col * 4)), y);
          else
            store_out<4 * CT>(reinterpret_cast<uint16_t *>(rows + (token * so + col * 2)), y);
        };
        if (r == C) {
#pragma unroll
          for (int it = 0; it < IT; ++it) put(it);
        } else {
#pragma unroll
          for (int it = 0; it < IT; ++it)
            if (16 * it + c < r) put(it);
        }
      }

      // state
      const float carry = lds.pw[r];
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) S[kt][ct] *= carry;
#pragma unroll
      for (int js = 0; js < JS; ++js) {
        typename O::frag wf[CT][O::kValueParts];
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
          float x[8];
          O::expand(vf[js][ct], x);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] *= lds.upd[C - r + 32 * js + 8 * g + e];
          O::parts(x, wf[ct]);
        }
#pragma unroll
        for (int k4 = 0; k4 < KT; k4 += 4) {
          typename O::frag kf[4];
#pragma unroll
          for (int m = 0; m < 4; ++m)
            kf[m] = O::cols(lds.k, L::ldk, 32 * js, 32 * ((k4 + m) / 2) + 4 * (m % 2), 8, lane);
#pragma unroll
          for (int n2 = 0; n2 < O::kValueParts; ++n2) {
            if (n2 == 2 && !exact) break;
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
              for (int ct = 0; ct < CT; ++ct)
                S[k4 + m][ct] = O::mma(kf[m], wf[ct][n2], S[k4 + m][ct]);
          }
        }
      }
    }

    if constexpr (OUTPUT) {
      if (done_here && R.final_state && slot >= 0) store_state(R.final_state, slot);
      if (!p.window) break;
    } else {
      store_state(R.carried, place);
      break;
    }
  }
}

// The states at the borders from the windows' sums, four elements per thread, in place.
// The chain along the borders is a multiply-add each; the loads of 16 borders are in flight
// together (15 borders of 32 heads, 64 KB each: 7.3 us; eight at a time in
// workgroups of four waves 10.5 us).
constexpr int kCombineThreads = 64;
__global__ void __launch_bounds__(kCombineThreads)
    linear_combine_kernel(const LinearParams p, long size4) {
  const LinearRole &R = p.role[blockIdx.y];
  const long i = static_cast<long>(blockIdx.x) * kCombineThreads + threadIdx.x;
  const float w = decay_power(p.g[i / size4], p.window);
  if (w == 0.0f) return;   // no sum reaches past its own border
  float4 *at = reinterpret_cast<float4 *>(R.carried) + i;
  const long stride = size4 * p.H;
  const int borders = p.windows - 1;
  constexpr int kAhead = 16;
  float4 H = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int s = 0; s < borders; s += kAhead) {
    float4 x[kAhead];
    int kind[kAhead];
#pragma unroll
    for (int m = 0; m < kAhead; ++m) {
      const int b = min(s + m, borders - 1), e = R.reverse ? borders - 1 - b : b;
      x[m] = at[e * stride];
      kind[m] = R.crossing[e];
    }
#pragma unroll
    for (int m = 0; m < kAhead; ++m) {
      if (s + m >= borders) break;
      const int e = R.reverse ? borders - 1 - (s + m) : s + m;
      if (kind[m] == 2) {
        H.x = fmaf(w, H.x, x[m].x);
        H.y = fmaf(w, H.y, x[m].y);
        H.z = fmaf(w, H.z, x[m].z);
        H.w = fmaf(w, H.w, x[m].w);
        at[e * stride] = H;
      } else {
        H = x[m];
      }
    }
  }
}

// gradients of a q/k head (dq, then dk): the sum of its value heads' parts, four channels
// per thread, as they stream by.  The parts are float32 and added in the heads' order, so
// that grouped heads cost no rounding and no atomics (1501 tokens of 4 on 2 heads of 64:
// 4.0 us, a launch's least; two launches 3.8 us each).
template <typename T>
__global__ void __launch_bounds__(256)
    sum_heads_kernel(const float *dq_parts, const float *dk_parts, T *dq, T *dk, long n4, int d4,
                     int group, int heads, const int32_t *end) {
  const float *in = blockIdx.y ? dk_parts : dq_parts;
  T *out = blockIdx.y ? dk : dq;
  const long i = static_cast<long>(blockIdx.x) * 256 + threadIdx.x;
  const long row = i / d4;   // token and q/k head
  if (i >= n4 || (end && row >= static_cast<long>(*end) * heads)) return;
  const float4 *src = reinterpret_cast<const float4 *>(in) + row * group * d4 + i % d4;
  float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int m = 0; m < group; ++m) {
    const float4 x = src[static_cast<long>(m) * d4];
    y[0] += x.x;
    y[1] += x.y;
    y[2] += x.z;
    y[3] += x.w;
  }
  store_out<4>(out + 4 * i, y);
}

// ---- decode ---------------------------------------------------------------------------
// One workgroup per (request, value head); thread t owns four value columns in every
// (256 / (V/4))-th key row, so the state sits in registers between its read and its write,
// which are all the traffic.  S' = lambda S + k v^T, then o = scale q S'.
// 128 requests (112 live) of 32 heads of 128 x 128: 475 MB in 97 us, 4.9 TB/s, what a large
// copy reaches; one request 4.8 us, the trip to memory and back, of 10.7 us that the host
// takes to call it.
template <typename T, typename TOut, int DK, int DV>
__global__ void __launch_bounds__(256) linear_decode_kernel(const LinearDecodeParams p) {
  constexpr int CG = DV / 4, RG = 256 / CG, RPT = DK / RG;
  __shared__ float ks[DK], qs[DK];
  __shared__ float red[4][DV];
  const int i = blockIdx.x / p.Hv, h = blockIdx.x % p.Hv, hk = h / (p.Hv / p.Hk);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int cg = tid % CG, rg = tid / CG;
  const int r = p.batch_indices ? p.batch_indices[i] : i;
  const size_t state_size = static_cast<size_t>(DK) * DV;
  float *st = p.state + (static_cast<size_t>(r < 0 ? 0 : r) * p.Hv + h) * state_size;
  float4 H[RPT];
#pragma unroll
  for (int m = 0; m < RPT; ++m)
    H[m] = *reinterpret_cast<const float4 *>(st + static_cast<size_t>(rg + RG * m) * DV + 4 * cg);
  const float lam = expf(p.g[h]);
  auto store_state = [&](float *dst) {
#pragma unroll
    for (int m = 0; m < RPT; ++m)
      *reinterpret_cast<float4 *>(dst + static_cast<size_t>(rg + RG * m) * DV + 4 * cg) = H[m];
  };
  for (int t = 0; t < p.num_tokens; ++t) {
    const size_t tok = static_cast<size_t>(i) * p.num_tokens + t;
    const T *src = static_cast<const T *>(wave & 1 ? p.q : p.k) + (tok * p.Hk + hk) * DK;
    if (wave < 2)
      for (int e = lane; e < DK; e += 64) (wave & 1 ? qs : ks)[e] = load_f32(src + e);
    const T *vg = static_cast<const T *>(p.v) + (tok * p.Hv + h) * DV + 4 * cg;
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = load_f32(vg + e);
    __syncthreads();
    float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int m = 0; m < RPT; ++m) {
      const float kv = ks[rg + RG * m], qv = qs[rg + RG * m];
      H[m].x = fmaf(kv, v[0], lam * H[m].x);
      H[m].y = fmaf(kv, v[1], lam * H[m].y);
      H[m].z = fmaf(kv, v[2], lam * H[m].z);
      H[m].w = fmaf(kv, v[3], lam * H[m].w);
      y[0] = fmaf(qv, H[m].x, y[0]);
      y[1] = fmaf(qv, H[m].y, y[1]);
      y[2] = fmaf(qv, H[m].z, y[2]);
      y[3] = fmaf(qv, H[m].w, y[3]);
    }
#pragma unroll
    for (int o = CG; o < 64; o <<= 1)
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] += __shfl_xor(y[e], o);
    if (lane < CG)
      *reinterpret_cast<float4 *>(&red[wave][4 * cg]) = make_float4(y[0], y[1], y[2], y[3]);
    __syncthreads();
    if (tid < DV)
      store_f32(static_cast<TOut *>(p.out) + (tok * p.Hv + h) * DV + tid,
                p.scale * (red[0][tid] + red[1][tid] + red[2][tid] + red[3][tid]));
    if (p.intermediate_state && r >= 0)
      store_state(p.intermediate_state + (tok * p.Hv + h) * state_size);
  }
  if (r >= 0) store_state(st);   // padding writes no state
}

template <typename T, bool OUTPUT>
hipError_t launch_dims(LinearParams p, int dq, int dv, hipStream_t s) {
  const long places = linear_places(p, OUTPUT);
  // A head's 128 value columns go to two workgroups where one each would not give every
  // compute unit two: half the products per chunk for one more pass over q and k (2 x 1023
  // tokens of 4 heads in float32, 128 workgroups: 36.0 us whole, 29.0 halved; 240 tokens of
  // 64 heads in bf16, 64: 28.8 and 22.5; 16383 tokens of 16 heads in bf16, 512: 129 and 149).
  p.halves = dv == 128 && places * p.H * p.roles <= 256;
  if (p.halves) dv = 64;
  const long sets = (places * p.Hk + 7) / 8 * 8;   // whole rounds over the XCDs
  const dim3 grid(static_cast<unsigned>((sets * p.roles * p.group) << p.halves));
  const dim3 block(threads(dv, OUTPUT));
  if (dq == 128 && dv == 128)
    hipLaunchKernelGGL((linear_attention_kernel<T, 128, 128, OUTPUT>), grid, block, 0, s, p);
  else if (dq == 128)
    hipLaunchKernelGGL((linear_attention_kernel<T, 128, 64, OUTPUT>), grid, block, 0, s, p);
  else if (dv == 128)
    hipLaunchKernelGGL((linear_attention_kernel<T, 64, 128, OUTPUT>), grid, block, 0, s, p);
  else
    hipLaunchKernelGGL((linear_attention_kernel<T, 64, 64, OUTPUT>), grid, block, 0, s, p);
  return hipGetLastError();
}

template <typename T, typename TOut>
hipError_t decode_dims(const LinearDecodeParams &p, int dk, int dv, hipStream_t s) {
  const dim3 grid(p.batch * p.Hv), block(256);
  if (dk == 128 && dv == 128)
    hipLaunchKernelGGL((linear_decode_kernel<T, TOut, 128, 128>), grid, block, 0, s, p);
  else if (dk == 128)
    hipLaunchKernelGGL((linear_decode_kernel<T, TOut, 128, 64>), grid, block, 0, s, p);
  else if (dv == 128)
    hipLaunchKernelGGL((linear_decode_kernel<T, TOut, 64, 128>), grid, block, 0, s, p);
  else
    hipLaunchKernelGGL((linear_decode_kernel<T, TOut, 64, 64>), grid, block, 0, s, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_attention(const LinearParams &p, int in_f32, int dq, int dv,
                                   hipStream_t stream) {
  return in_f32 ? launch_dims<float, true>(p, dq, dv, stream)
                : launch_dims<uint16_t, true>(p, dq, dv, stream);
}

hipError_t launch_linear_borders(const LinearParams &p, int in_f32, int dq, int dv,
                                 hipStream_t stream) {
  const hipError_t e = in_f32 ? launch_dims<float, false>(p, dq, dv, stream)
                              : launch_dims<uint16_t, false>(p, dq, dv, stream);
  if (e != hipSuccess) return e;
  const long size4 = static_cast<long>(dq) * dv / 4;
  const dim3 grid(static_cast<unsigned>(size4 * p.H / kCombineThreads), p.roles);
  hipLaunchKernelGGL(linear_combine_kernel, grid, dim3(kCombineThreads), 0, stream, p, size4);
  return hipGetLastError();
}

int linear_window(long tokens, int heads, int num_seqs, int packed, int roles) {
  // Workgroups wanted: two per compute unit, as many as are resident; the three roles of the
  // backward have 256 each, one round and a half (packed prefill of 36112 tokens, 32 heads: 256
  // places 512 us, 512 422, 1024 440; one prompt of 16383 tokens, 16 heads: 137, 129, 154;
  // backward of 4 x 4096 tokens, 16 heads: 128 places 311, 256 270, 512 282).
  const long places = roles > 1 ? 256 : 512;
  if (tokens <= 256 || (!packed && static_cast<long>(num_seqs) * heads >= places)) return 0;
  const long windows = (places + heads - 1) / heads;
  const long window = ((tokens + windows - 1) / windows + 63) / 64 * 64;
  return static_cast<int>(window >= tokens ? 0 : window);
}

hipError_t launch_sum_heads(const float *dq_parts, const float *dk_parts, void *dq, void *dk,
                            long rows, int d, int group, int heads, const int32_t *end,
                            int out_f32, hipStream_t stream) {
  const long n4 = rows * d / 4;
  if (n4 == 0) return hipSuccess;
  const dim3 grid(static_cast<unsigned>((n4 + 255) / 256), 2), block(256);
  if (out_f32)
    hipLaunchKernelGGL((sum_heads_kernel<float>), grid, block, 0, stream, dq_parts, dk_parts,
                       static_cast<float *>(dq), static_cast<float *>(dk), n4, d / 4, group, heads,
                       end);
  else
    hipLaunchKernelGGL((sum_heads_kernel<uint16_t>), grid, block, 0, stream, dq_parts, dk_parts,
                       static_cast<uint16_t *>(dq), static_cast<uint16_t *>(dk), n4, d / 4, group,
                       heads, end);
  return hipGetLastError();
}

hipError_t launch_linear_decode(const LinearDecodeParams &p, int in_f32, int out_f32, int dk, int dv,
                                hipStream_t stream) {
  if (in_f32)
    return out_f32 ? decode_dims<float, float>(p, dk, dv, stream)
                   : decode_dims<float, uint16_t>(p, dk, dv, stream);
  return out_f32 ? decode_dims<uint16_t, float>(p, dk, dv, stream)
                 : decode_dims<uint16_t, uint16_t>(p, dk, dv, stream);
}

}  // namespace gdr
