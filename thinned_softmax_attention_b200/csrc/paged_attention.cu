// Attention of single query tokens over lists of cache pages, split over the keys and joined.
//
//   z_j = s q.k_j log2 e,  m = max z,  l = sum 2^(z_j - m),  o = sum 2^(z_j - m) v_j / l
// A key head's G query rows share its keys, so each key and value row is read once and used for G dot
// products: about 2 G FLOP per byte, far below the machine's balance.  HBM bounds it; everything below
// serves to keep enough reads in flight and the tail short.
//
// Work.  The keys of (token, key head) pairs, token by token, form one line of units of
// 16 keys per warp.  Every CTA of a fixed grid takes an equal stretch of that line, whatever the
// lengths are (they are only known on the device): long requests are split, short ones
// packed.  A pair that lies in one CTA is finished there; one that is cut leaves a partial (m, l, o)
// per CTA, and the join kernel, launched behind it, adds up those of each cut pair.
//
// Reads.  A warp owns a ring of stages in shared memory, 16 keys and values each, filled by its own
// asynchronous copies (no barrier of the CTA in the loop): the ring runs on across pairs, so the next
// pair's keys arrive while this one is joined.  The page ids are fetched a step ahead.  Rows that
// are not seen (behind the length, before the window, on a page outside the pool) are filled with zeros, so that
// nothing stored there, NaN or not, meets a weight of zero.
//
// Products (16-bit and 8-bit caches), mma m16n8k16: S = Q K^T with the rows of Q as M, O += P V.  The
// order of the summed index is free, so a lane takes its B fragments of K as whole 16-byte pieces of
// a row, and the column order of S is chosen so that S's accumulator is P's A fragment as it stands:
// lane (r, c) holds the columns of keys 4 c .. 4 c + 3, reads those four rows of V as 16-byte pieces
// (of d = DC (r + 8 i) ..) and pairs them up with byte permutations.  No transposing load, no shuffle but
// the row maximum.  G <= 8 leaves the tile's upper 8 rows free: they carry P's rounding error, so P
// keeps 16 bits and more at no cost; G <= 16 issues that product separately (bf16 against e4m3: none, kSplit).
//
// fp32 caches use the tf32 products (m16n8k8) with every operand as the sum of two tf32 numbers,
// (a_hi + a_lo)(b_hi + b_lo), good to 2^-22.  The upper rows of the tile carry a_lo, so that takes two products.
//
// The tensor cores cut their sums, they do not round them: a sum that runs on in an accumulator drifts towards
// zero, by 2.5e-4 over 65536 keys of a CTA in fp32, by 1e-4 in the 16-bit types.  So the products of P and V begin at zero
// every 16 keys (fp32: 8), as those of fp32's scores do every 32 columns, and are added up by ordinary additions, which
// take the rescaling with the maximum along.  That costs 3% (e4m3) or nothing seen (16 bits; 16 rows of width 256: -8%).
//
// These are the 16-row products on purpose: tcgen05 tiles have 64 or 128 rows, of which G would fill a few,
// and their operands pass through shared memory in fixed layouts, P included.  The tensor pipe is no bound here
// (32% busy at e4m3, the densest case of up to 8 rows; issue slots 52%).
//
// B200 (copy rate 6.46 TB/s), width 128, bf16, 4 query rows to a key head unless stated:
//   16 requests of 65536 .. 131072 keys, 8 heads     0.89 .. 0.95 ms   7.0 .. 6.6 TB/s
//   48 requests of 1 .. 8192 keys, 8 heads           54 us             5.5 TB/s     16 query rows: 64 us
//   40 requests of 32768 keys, 4 heads, e4m3         0.23 ms           5.8 TB/s     16 query rows: 0.25, fp16 0.32 ms
//   16 requests of 32768 .. 65536 keys, fp32         1.32 ms           4.8 TB/s     width 256, 48 of 8192: 3.5 TB/s
//   1 request of 500 keys, 32 heads                  9.8 us            (6.4 of them with 64 keys)
// What is left of the first three is the 10 us at the ends: launch, lengths, first reads, join.  In fp32 it is the splitting
// of every key and value into its two parts, and at width 256 one CTA per SM with two short stages.
#include <type_traits>

#include "paged.h"
#include "paged_types.cuh"

namespace thin {

namespace {

constexpr int kAlign = 32;         // keys before a window that its first stage may hold, a multiple of a stage's
constexpr int kMaxCtas = 444;      // 148 SMs x 3

// One token of the call: its row of outputs, its visible keys [start, len) and their units.
struct Token {
  int len, start, units;
  const int32_t* ids;
  bool live;   // not padding
};

// key / page for key < 2^31, page <= 65536: by the reciprocal that the host rounded up (PagedAttn).
__device__ __forceinline__ int page_of(const PagedAttn& p, int key) {
  return p.page_mul ? (int)(__umulhi((uint32_t)key, p.page_mul) >> p.page_shift) : key;
}

template <int UNIT>
__device__ __forceinline__ Token token_from(const PagedAttn& p, int n, int row, int len) {
  Token t;
  t.live = row >= 0 && row < p.a.R;
  t.len = t.live ? min(max(len, 0), p.list_width * p.a.page) : 0;
  t.start = p.a.window && t.len > p.a.window ? t.len - p.a.window : 0;
  const int first = t.start & ~(kAlign - 1);
  t.units = (t.len - first + UNIT - 1) / UNIT;
  t.ids = p.ids + (p.list_rows ? row : n) * p.ids_token;
  return t;
}
template <int UNIT>
__device__ __forceinline__ Token token_of(const PagedAttn& p, int n) {
  return token_from<UNIT>(p, n, p.a.rows ? p.a.rows[n] : n, p.keys[n]);
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool full) {
  const int n = full ? 16 : 0;   // the rest is filled with zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ void sts16(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A sum of leading parts and what their lower parts add: nothing where it is infinite, since a lower part of 0
// or of the other sign makes a NaN of an infinite factor.
__device__ __forceinline__ float with_rest(float lead, float rest) { return fabsf(lead) == INFINITY ? lead : lead + rest; }

template <typename M>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  uint32_t r;
  if constexpr (std::is_same<M, __nv_bfloat16>::value)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
// The same, cut instead of rounded.
template <typename M>
__device__ __forceinline__ uint32_t pack2_cut(float a, float b) {
  uint32_t r;
  if constexpr (std::is_same<M, __nv_bfloat16>::value)
    asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  else
    asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
template <typename M>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (std::is_same<M, __nv_bfloat16>::value)
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  else
    return __half22float2(*(const __half2*)&w);
}
template <typename M>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<M, __nv_bfloat16>::value)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Four e4m3 values as fp16 ones (exact), two to a word.
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{ .reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; cvt.rn.f16x2.e4m3x2 %1, h; }" : "=r"(lo), "=r"(hi) : "r"(w));
}

// ---------------------------------------------------------------------------------------------
// One warp's part of a tile of ROWS query rows, on the tensor cores.
// ---------------------------------------------------------------------------------------------
template <typename T, typename C, int HD, int ROWS_>
struct MmaTile {
  static constexpr int ROWS = ROWS_;
  static constexpr int COLS = ROWS == 8 && HD > 64 ? 128 : 64;   // columns joined at a time
  static constexpr int kSmem = 0;
  static constexpr bool k8 = sizeof(C) == 1;
  using M = typename std::conditional<k8, __half, T>::type;   // the products' type
  static constexpr int RB = HD * (int)sizeof(C);              // bytes of a stage's row
  static constexpr int DC = 16 / (int)sizeof(C);              // elements of a 16-byte piece
  static constexpr int KJ = RB / 64, VI = RB / 128;           // pieces of K and V per lane and row
  static constexpr int QW = DC / 2;                           // words of Q per piece
  // P as two numbers.  One is enough for 16 bf16 rows against e4m3: off by 2^-11 at most, an eighth of what the output is
  // rounded by; the second product would take 252 us to 299 (40 requests of 32768 keys; fp16 282 to 320)
  static constexpr bool kSplit = !k8 || ROWS == 8 || std::is_same<T, __half>::value;
  static constexpr int kKeys = RB <= 128 ? 32 : 16;           // keys of a stage: short rows, twice as many for the same overhead
  static constexpr int NB = kKeys / 16;                       // products' blocks of 16 keys
  // fp16 weights are lifted by 2^14: without that those below 2^-14 of the largest lose bits, and a long
  // tail of keys at 2^-25 is rounded up or away as a whole
  static constexpr float kLift = std::is_same<M, __half>::value ? 16384.f : 1.f;
  // With 16 rows one sum takes both parts' products, and an infinite value must meet two parts of one sign: the leading
  // one is cut, and the lower one is made positive, in bf16 by the weight's last bit, in fp16 by the least step.  (Leaving
  // infinities out of the lower product instead took 5% to 10%; e4m3 has none.)
  static constexpr bool kOneSign = ROWS == 16 && !k8;
  static_assert(ROWS == 8 || ROWS == 16, "");
  static_assert(VI >= 1 && KJ == 2 * VI, "");

  // Rows of a stage lie one behind the other; the 16-byte pieces of a row are permuted within groups of
  // eight so that the fragment reads below meet every bank once: K's quarter-warps read the same pieces of two
  // neighbouring rows, V's two neighbouring pieces of rows 4 apart.
  static __device__ __forceinline__ int swizzle(int row) { return ((row & 1) << 2) ^ (((row >> 2) & 3) << 1); }

  uint32_t q[KJ][ROWS / 8][QW], next[KJ][ROWS / 8][QW];
  float o[VI][DC][4];
  float m[2], l[2], sc[2];

  // Query rows are fetched a step before the pair that they belong to, where the registers allow it.
  static constexpr bool kAhead = HD <= 128 && !k8;
  __device__ __forceinline__ void fetch(const PagedAttn& p, int n, int row0, int rows, int lane) {
    const int r = lane >> 2, c = lane & 3;
#pragma unroll
    for (int x = 0; x < ROWS / 8; ++x) {
      const int g = r + 8 * x;
      const T* src = (const T*)p.a.q + n * p.a.q_token + (row0 + g) * p.a.q_head;
#pragma unroll
      for (int j = 0; j < KJ; ++j) {
        const int e = (c + 4 * j) * DC;
#pragma unroll
        for (int y = 0; y < QW; y += 4) {
          uint4 u = make_uint4(0, 0, 0, 0);
          if (g < rows && e < p.a.E) u = ((const uint4*)(src + e))[y / 4];
          next[j][x][y] = u.x;
          next[j][x][y + 1] = u.y;
          next[j][x][y + 2] = u.z;
          next[j][x][y + 3] = u.w;
        }
      }
    }
  }

  // bf16 queries as fp16 by way of shared memory: 16-byte loads leave them in neighbouring registers, where conversions
  // spilled 64 of them (40 e4m3 requests of width 256: 75 us, without 120; of width 128, which does not spill, 43.0, without 42.0)
  static constexpr bool kByShared = HD == 256 && ROWS == 8;
  // own: the warp's part of the merge buffer, which no other warp uses between two pairs' ends
  __device__ __forceinline__ void reset(const PagedAttn& p, int n, int row0, int rows, float scale, int lane, float* own) {
    static_assert(!kByShared || KJ * QW * 128 <= ROWS * COLS * 4, "");
    if constexpr (!kAhead) fetch(p, n, row0, rows, lane);
#pragma unroll
    for (int x = 0; x < ROWS / 8; ++x) {
      sc[x] = scale;
      if constexpr (k8 && !std::is_same<T, __half>::value) {
        // q into fp16, times the power of two that brings the row's largest value to 2^13 .. 2^14: its eight bits
        // stay whole down to 2^-30 of that (where it lies below 2^-113, the power stops at 126: down to 2^-143)
        float mx = 0.f;
#pragma unroll
        for (int j = 0; j < KJ; ++j)
#pragma unroll
          for (int y = 0; y < QW; ++y) {
            const float2 f = unpack2<T>(next[j][x][y]);
            mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
          }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const int up = min(140 - (int)(__float_as_uint(mx) >> 23), 126);   // -115 for infinities
#pragma unroll
        for (int j = 0; j < KJ; ++j)
#pragma unroll
          for (int y = 0; y < QW; ++y) {
            const float2 f = unpack2<T>(next[j][x][y]);
            next[j][x][y] = pack2<__half>(f.x * pow2f(up), f.y * pow2f(up));
          }
        const uint32_t at = (uint32_t)__cvta_generic_to_shared(own) + lane * 16;
#pragma unroll
        for (int j = 0; j < KJ; ++j)
#pragma unroll
          for (int y = 0; y < QW; y += 4) {
            uint4 u = make_uint4(next[j][x][y], next[j][x][y + 1], next[j][x][y + 2], next[j][x][y + 3]);
            if constexpr (kByShared) {
              sts16(at + (j * QW + y) * 128, u);
              u = lds16(at + (j * QW + y) * 128);
            }
            q[j][x][y] = u.x;
            q[j][x][y + 1] = u.y;
            q[j][x][y + 2] = u.z;
            q[j][x][y + 3] = u.w;
          }
        sc[x] = scale * pow2f(-up);
      } else {
#pragma unroll
        for (int j = 0; j < KJ; ++j)
#pragma unroll
          for (int y = 0; y < QW; ++y) q[j][x][y] = next[j][x][y];
      }
      m[x] = -INFINITY;
      l[x] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < VI; ++i)
#pragma unroll
      for (int y = 0; y < DC; ++y) o[i][y][0] = o[i][y][1] = o[i][y][2] = o[i][y][3] = 0.f;
  }

  // One stage: keys at smem address ks, values at vs; bit j of `seen` is key j's.
  __device__ __forceinline__ void step(const PagedAttn& p, uint32_t ks, uint32_t vs, uint32_t seen, int lane, float*) {
    const int r = lane >> 2, c = lane & 3;
    float s[NB][2][4] = {}, s2[NB][2][4] = {};   // two chains per tile, for the products' latency
    const uint32_t zero = 0;
    // column r of S's tile t is key 4 (r >> 1) + 2 t + (r & 1) of a block
    const uint32_t ka = ks + (4 * (r >> 1) + (r & 1)) * RB + ((c ^ swizzle(4 * (r >> 1) + (r & 1))) << 4);
#pragma unroll
    for (int j = 0; j < KJ; ++j) {
      if (j * 4 * DC >= p.a.E) break;
#pragma unroll
      for (int t = 0; t < 2 * NB; ++t) {
        const uint4 u = lds16((ka ^ ((j & 1) << 6)) + ((t >> 1) * 16 + 2 * (t & 1)) * RB + (j >> 1) * 128);
        uint32_t b[QW];
        if constexpr (k8) {
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int y = 0; y < 4; ++y) widen4(w[y], b[2 * y], b[2 * y + 1]);
        } else {
          b[0] = u.x;
          b[1] = u.y;
          b[2] = u.z;
          b[3] = u.w;
        }
#pragma unroll
        for (int y = 0; y < QW; y += 2) {
          const uint32_t a[4] = {q[j][0][y], ROWS == 16 ? q[j][ROWS / 8 - 1][y] : zero, q[j][0][y + 1],
                                 ROWS == 16 ? q[j][ROWS / 8 - 1][y + 1] : zero};
          mma<M>(y & 2 ? s2[t >> 1][t & 1] : s[t >> 1][t & 1], a, b[y], b[y + 1]);
        }
      }
    }
    // s[b][t][2 x + u] = row r + 8 x against key 16 b + 4 c + 2 t + u; z is rounded before the maximum is taken,
    // so that z - m is 0 at the maximum, however large both are
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int x = 0; x < ROWS / 8; ++x) {
          s[b][t][2 * x] = (s[b][t][2 * x] + s2[b][t][2 * x]) * sc[x];
          s[b][t][2 * x + 1] = (s[b][t][2 * x + 1] + s2[b][t][2 * x + 1]) * sc[x];
        }
    if (seen != (kKeys == 32 ? 0xFFFFFFFFu : 0xFFFFu)) {
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int u = 0; u < 2; ++u)
            if (!((seen >> (16 * b + 4 * c + 2 * t + u)) & 1)) s[b][t][u] = s[b][t][2 + u] = -INFINITY;
    }
    uint32_t hi[2][NB][2], lo[2][NB][2];   // [x][b][t]
    float f[2];
#pragma unroll
    for (int x = 0; x < ROWS / 8; ++x) {
      float mx = -INFINITY;
#pragma unroll
      for (int b = 0; b < NB; ++b)
        mx = fmaxf(mx, fmaxf(fmaxf(s[b][0][2 * x], s[b][0][2 * x + 1]), fmaxf(s[b][1][2 * x], s[b][1][2 * x + 1])));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float mn = fmaxf(m[x], mx);
      const float ref = mn == -INFINITY ? 0.f : mn;
      f[x] = ex2(m[x] - ref);
      m[x] = mn;
      float sum = 0.f;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const float p0 = ex2(s[b][t][2 * x] - ref), p1 = ex2(s[b][t][2 * x + 1] - ref);
          sum += p0 + p1;
          float w0 = p0 * kLift, w1 = p1 * kLift;
          if constexpr (kOneSign && std::is_same<M, __nv_bfloat16>::value) {
            w0 = __uint_as_float(__float_as_uint(w0) | 1u);
            w1 = __uint_as_float(__float_as_uint(w1) | 1u);
          }
          hi[x][b][t] = kOneSign ? pack2_cut<M>(w0, w1) : pack2<M>(w0, w1);
          if constexpr (kSplit) {
            const float2 h = unpack2<M>(hi[x][b][t]);
            lo[x][b][t] = pack2<M>(w0 - h.x, w1 - h.y);
          }
          if constexpr (kOneSign && std::is_same<M, __half>::value) {
            const __half2 least = __hmin2(*(const __half2*)&hi[x][b][t], __half2half2(__ushort_as_half(1)));   // 0 where the weight is
            *(__half2*)&lo[x][b][t] = __hmax2(*(const __half2*)&lo[x][b][t], least);
          }
        }
      l[x] = l[x] * f[x] + sum;
    }
    const float f1 = ROWS == 16 ? f[ROWS / 8 - 1] : f[0];
    auto add = [&](float (&x)[4], const float (&t)[4], int b) {
#pragma unroll
      for (int z = 0; z < 4; ++z) x[z] = b ? x[z] + t[z] : fmaf(x[z], z < 2 ? f[0] : f1, t[z]);
    };
    const uint32_t va = vs + 4 * c * RB + ((r ^ (c << 1)) << 4);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const uint32_t a[4] = {hi[0][b][0], ROWS == 16 ? hi[ROWS / 8 - 1][b][0] : lo[0][b][0], hi[0][b][1],
                             ROWS == 16 ? hi[ROWS / 8 - 1][b][1] : lo[0][b][1]};
      const uint32_t a2[4] = {lo[0][b][0], lo[ROWS / 8 - 1][b][0], lo[0][b][1], lo[ROWS / 8 - 1][b][1]};
#pragma unroll
      for (int i = 0; i < VI; ++i) {
        if (i * 8 * DC >= p.a.D) break;
        uint32_t v[4][4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint4 u = lds16((va ^ ((k & 1) << 6)) + (16 * b + k) * RB + i * 128);   // swizzle(4 c + k) = 4 (k & 1) ^ 2 c
          v[k][0] = u.x;
          v[k][1] = u.y;
          v[k][2] = u.z;
          v[k][3] = u.w;
        }
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          if constexpr (k8) {
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              // bytes 2 y and 2 y + 1 of the word, those of two keys side by side
              const uint32_t b0 = __byte_perm(v[0][w], v[1][w], y ? 0x7362 : 0x5140);
              const uint32_t b1 = __byte_perm(v[2][w], v[3][w], y ? 0x7362 : 0x5140);
              uint32_t p0[2], p1[2];
              widen4(b0, p0[0], p0[1]);
              widen4(b1, p1[0], p1[1]);
              float t0[4] = {}, t1[4] = {};
              if constexpr (kSplit && ROWS == 16) {
                mma<M>(t0, a2, p0[0], p1[0]);
                mma<M>(t1, a2, p0[1], p1[1]);
              }
              mma<M>(t0, a, p0[0], p1[0]);
              mma<M>(t1, a, p0[1], p1[1]);
              add(o[i][4 * w + 2 * y], t0, b);
              add(o[i][4 * w + 2 * y + 1], t1, b);
            }
          } else {
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const uint32_t sel = y ? 0x7632 : 0x5410;
              const uint32_t b0 = __byte_perm(v[0][w], v[1][w], sel), b1 = __byte_perm(v[2][w], v[3][w], sel);
              float t[4] = {};
              if constexpr (ROWS == 16) mma<M>(t, a2, b0, b1);
              mma<M>(t, a, b0, b1);
              add(o[i][2 * w + y], t, b);
            }
          }
        }
      }
    }
  }

  // The sums over the lanes of a row; then (m, l) of row g at ml[2 g].
  __device__ __forceinline__ void finish(float* ml, int lane) {
#pragma unroll
    for (int x = 0; x < ROWS / 8; ++x) {
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
      if ((lane & 3) == 0) {
        ml[2 * ((lane >> 2) + 8 * x)] = m[x];
        ml[2 * ((lane >> 2) + 8 * x) + 1] = l[x];
      }
    }
  }
  // Columns [COLS part, COLS part + COLS) of o into dst (ROWS x COLS).
  static __device__ __forceinline__ int place(int g, int col) {   // float4 `col` of row g: quarter-warps meet every bank once
    return g * (COLS / 4) + (col ^ ((col >> 3) & 3) ^ ((g & 1) << (k8 ? 2 : 1)));
  }
  __device__ __forceinline__ void put(float4* dst, int part, int lane) {
    const int r = lane >> 2, c = lane & 3;
#pragma unroll
    for (int i = 0; i < VI; ++i)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int d = DC * (2 * c + u + 8 * i);
        if (d / COLS != part) continue;
#pragma unroll
        for (int y = 0; y < DC; y += 4) {
          const int col = (d % COLS + y) / 4;
          constexpr float by = 1.f / kLift;
          if constexpr (ROWS == 8) {
            dst[place(r, col)] = make_float4(with_rest(o[i][y][u], o[i][y][2 + u]) * by, with_rest(o[i][y + 1][u], o[i][y + 1][2 + u]) * by,
                                             with_rest(o[i][y + 2][u], o[i][y + 2][2 + u]) * by, with_rest(o[i][y + 3][u], o[i][y + 3][2 + u]) * by);
          } else {
            dst[place(r, col)] = make_float4(o[i][y][u] * by, o[i][y + 1][u] * by, o[i][y + 2][u] * by, o[i][y + 3][u] * by);
            dst[place(r + 8, col)] =
                make_float4(o[i][y][2 + u] * by, o[i][y + 1][2 + u] * by, o[i][y + 2][2 + u] * by, o[i][y + 3][2 + u] * by);
          }
        }
      }
  }
};

// ---------------------------------------------------------------------------------------------
// The same for fp32.
// ---------------------------------------------------------------------------------------------
// x = hi + lo, hi rounded to the 11 bits of tf32; of lo's 12 bits and a sign the product takes the leading
// 11, so what is lost is at most 2^-23 of x's leading bit.
struct Split {
  uint32_t hi[4], lo[4];
};
__device__ __forceinline__ Split split4(uint4 u) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  Split s;
  float mx = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s.hi[i] = (w[i] + 0x1000u) & 0xFFFFE000u;
    s.lo[i] = __float_as_uint(__uint_as_float(w[i]) - __uint_as_float(s.hi[i]));
    mx = fmaxf(mx, fabsf(__uint_as_float(w[i])));
  }
  if (mx > 3.4e38f) {   // hi may not be rounded up to an infinity, and an infinity has no lower part
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s.hi[i] = w[i] & 0xFFFFE000u;
      s.lo[i] = (w[i] & 0x7FFFFFFFu) == 0x7F800000u ? 0u : __float_as_uint(__uint_as_float(w[i]) - __uint_as_float(s.hi[i]));
    }
  }
  return s;
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int HD>
struct Tf32Tile {
  static constexpr int ROWS = 8, kKeys = 8;
  static constexpr int RB = HD * 4;
  static constexpr int KJ = HD / 16, VI = HD / 32;
  static constexpr bool kAhead = false;
  static constexpr bool kQueryInSmem = HD > 128;   // the registers do not hold it beside o
  static constexpr int kSmem = kQueryInSmem ? 2 * ROWS * HD * 4 : 0;   // of the CTA: its parts hi and lo

  uint32_t qh[kQueryInSmem ? 1 : KJ][4], ql[kQueryInSmem ? 1 : KJ][4];
  float o[VI][4][4];
  float m, l, sc;

  // K's quarter-warps read the same pieces of two neighbouring rows, V's two neighbouring pieces of rows 2 apart.
  static __device__ __forceinline__ int swizzle(int row) { return ((row & 1) << 2) ^ (((row >> 1) & 3) << 1); }

  // piece `col` of row r of the queries in shared memory, as an index of uint4
  static __device__ __forceinline__ int query_at(int r, int col) { return r * (HD / 4) + (col ^ ((r & 1) << 2)); }

  __device__ __forceinline__ void reset(const PagedAttn& p, int n, int row0, int rows, float scale, int lane, float* sm) {
    const float* src = (const float*)p.a.q + n * p.a.q_token + row0 * p.a.q_head;
    if constexpr (kQueryInSmem) {   // for every thread of the CTA alike, and behind the last pair's join
      for (int i = threadIdx.x; i < ROWS * HD / 4; i += blockDim.x) {
        const int r = i / (HD / 4), col = i % (HD / 4);
        const Split s = split4(r < rows && col * 4 < p.a.E ? *(const uint4*)(src + r * p.a.q_head + col * 4) : make_uint4(0, 0, 0, 0));
        ((uint4*)sm)[query_at(r, col)] = make_uint4(s.hi[0], s.hi[1], s.hi[2], s.hi[3]);
        ((uint4*)sm)[ROWS * HD / 4 + query_at(r, col)] = make_uint4(s.lo[0], s.lo[1], s.lo[2], s.lo[3]);
      }
      __syncthreads();
    } else {
      const int r = lane >> 2, c = lane & 3;
#pragma unroll
      for (int j = 0; j < KJ; ++j) {
        const int e = (c + 4 * j) * 4;
        const Split s = split4(r < rows && e < p.a.E ? *(const uint4*)(src + r * p.a.q_head + e) : make_uint4(0, 0, 0, 0));
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          qh[j][y] = s.hi[y];
          ql[j][y] = s.lo[y];
        }
      }
    }
    sc = scale;
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int i = 0; i < VI; ++i)
#pragma unroll
      for (int y = 0; y < 4; ++y) o[i][y][0] = o[i][y][1] = o[i][y][2] = o[i][y][3] = 0.f;
  }

  __device__ __forceinline__ void step(const PagedAttn& p, uint32_t ks, uint32_t vs, uint32_t seen, int lane, float* sm) {
    const int r = lane >> 2, c = lane & 3;
    // products of the keys' leading parts and of their lower ones, 32 columns at a time (kChain)
    float s0[4] = {}, s1[4] = {}, s[4] = {};
    constexpr int kChain = 2;
    const uint32_t ka = ks + r * RB + ((c ^ swizzle(r)) << 4);   // column r of S is key r
#pragma unroll
    for (int j = 0; j < KJ; ++j) {
      if (j * 16 >= p.a.E) break;
      if (j && j % kChain == 0) {
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          s[y] += s0[y];
          s0[y] = 0.f;
        }
      }
      const Split k = split4(lds16((ka ^ ((j & 1) << 6)) + (j >> 1) * 128));
      uint32_t h[4], w[4];
      if constexpr (kQueryInSmem) {
        const uint4 qa = ((const uint4*)sm)[query_at(r, c + 4 * j)], qb = ((const uint4*)sm)[ROWS * HD / 4 + query_at(r, c + 4 * j)];
        h[0] = qa.x;
        h[1] = qa.y;
        h[2] = qa.z;
        h[3] = qa.w;
        w[0] = qb.x;
        w[1] = qb.y;
        w[2] = qb.z;
        w[3] = qb.w;
      } else {
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          h[y] = qh[j][y];
          w[y] = ql[j][y];
        }
      }
      const uint32_t a0[4] = {h[0], w[0], h[1], w[1]}, a1[4] = {h[2], w[2], h[3], w[3]};
      mma_tf32(s0, a0, k.hi[0], k.hi[1]);
      mma_tf32(s1, a0, k.lo[0], k.lo[1]);
      mma_tf32(s0, a1, k.hi[2], k.hi[3]);
      mma_tf32(s1, a1, k.lo[2], k.lo[3]);
    }
    // row r against keys 2 c and 2 c + 1; z is rounded before the maximum is taken, so that z - m is 0 at
    // the maximum, however large both are
    float z[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      z[u] = with_rest(s[u] + s0[u], (s[2 + u] + s0[2 + u]) + (s1[u] + s1[2 + u])) * sc;
      if (!((seen >> (2 * c + u)) & 1)) z[u] = -INFINITY;
    }
    float mx = fmaxf(z[0], z[1]);
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    const float mn = fmaxf(m, mx), ref = mn == -INFINITY ? 0.f : mn;
    const float f = ex2(m - ref);
    m = mn;
    // weights of 22 bits, which two tf32 numbers hold; the sum takes the same
    const float p0 = __uint_as_float(__float_as_uint(ex2(z[0] - ref)) & 0xFFFFFFFCu);
    const float p1 = __uint_as_float(__float_as_uint(ex2(z[1] - ref)) & 0xFFFFFFFCu);
    l = fmaf(l, f, p0 + p1);
    const uint32_t h0 = __float_as_uint(p0) & 0xFFFFE000u, h1 = __float_as_uint(p1) & 0xFFFFE000u;
    // P's slots c and c + 4 are keys 2 c and 2 c + 1
    const uint32_t a[4] = {h0, __float_as_uint(p0 - __uint_as_float(h0)), h1, __float_as_uint(p1 - __uint_as_float(h1))};
    const uint32_t va = vs + 2 * c * RB + ((r ^ (c << 1)) << 4);
#pragma unroll
    for (int i = 0; i < VI; ++i) {
      if (i * 32 >= p.a.D) break;
      const Split v0 = split4(lds16(va + i * 128)), v1 = split4(lds16((va ^ 64) + RB + i * 128));
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        float t[4] = {};
        mma_tf32(t, a, v0.lo[y], v1.lo[y]);
        mma_tf32(t, a, v0.hi[y], v1.hi[y]);
#pragma unroll
        for (int x = 0; x < 4; ++x) o[i][y][x] = fmaf(o[i][y][x], f, t[x]);
      }
    }
  }

  __device__ __forceinline__ void finish(float* ml, int lane) {
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    if ((lane & 3) == 0) {
      ml[2 * (lane >> 2)] = m;
      ml[2 * (lane >> 2) + 1] = l;
    }
  }
  static constexpr int COLS = HD == 128 ? 128 : 64;
  static __device__ __forceinline__ int place(int g, int col) { return g * (COLS / 4) + (col ^ (g & 1)); }
  __device__ __forceinline__ void put(float4* dst, int part, int lane) {
    const int r = lane >> 2, c = lane & 3;
#pragma unroll
    for (int i = 0; i < VI; ++i)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int d = 4 * (2 * c + u + 8 * i);
        if (d / COLS != part) continue;
        dst[place(r, d % COLS / 4)] = make_float4(with_rest(o[i][0][u], o[i][0][2 + u]), with_rest(o[i][1][u], o[i][1][2 + u]),
                                                  with_rest(o[i][2][u], o[i][2][2 + u]), with_rest(o[i][3][u], o[i][3][2 + u]));
      }
  }
};

// What a CTA leaves for the join kernel about the pair that begins in it and goes on behind it.
struct Cut {
  int n, tile, last, slot;   // token (-1: none), head tile, the CTA that it ends in, the partial's slot here
};
struct Parts {
  float* o;        // [2 grid][ROWS][D]
  float* ml;       // [2 grid][ROWS][2]
  Cut* cuts;       // [grid]
};

// A stage's place in the line, written by the warp that fills it.
struct alignas(16) Meta {
  int n, tile;     // tile: bit 30: the pair's first unit here, bit 31: its last one here
  uint32_t seen;   // a bit per key
  int left;        // units of the pair behind it
  __device__ __forceinline__ int which() const { return tile & 0x3FFFFFFF; }
  __device__ __forceinline__ bool first() const { return tile >> 30 & 1; }
  __device__ __forceinline__ bool last() const { return tile < 0; }
};

template <typename Tile, typename C, int HD, int WARPS, int STAGES>
struct Shape {
  static constexpr int kUnit = WARPS * Tile::kKeys;
  static constexpr int kStage = 2 * Tile::kKeys * HD * (int)sizeof(C);
  static constexpr int kRing = WARPS * STAGES * kStage;
  static constexpr int kMerge = WARPS * Tile::ROWS * Tile::COLS * 4;
  static constexpr int kSmem = kRing + kMerge + Tile::kSmem;
};

// A place on the line.
struct End {
  int n, tile, unit;
};

// A pair's stretch of the line: its units, and kPairCost more before them for what a pair costs besides
// its keys (the join of the warps, the outputs), in units.  Without them a stretch full of short
// requests takes several times as long as one within a long request (the 48 requests above: 0 units 101 us, 1 to
// 4 units 55 to 56; width 256: 1 unit 159, 2 units 122; width 64: 2 units 41, 4 units 43).
constexpr int kPairCost = 2;

template <typename Tile, typename T, typename C, int HD, int WARPS, int STAGES, int PER_SM>
__global__ void __launch_bounds__(WARPS * 32, PER_SM) attention_kernel(PagedAttn p, Parts parts) {
  using S = Shape<Tile, C, HD, WARPS, STAGES>;
  constexpr int ROWS = Tile::ROWS, RB = HD * (int)sizeof(C), kThreads = WARPS * 32, kKeys = Tile::kKeys;
  constexpr uint32_t kAll = kKeys == 32 ? 0xFFFFFFFFu : (1u << kKeys) - 1;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int64_t sums[WARPS];
  __shared__ End ends_s[2];
  __shared__ Meta meta[WARPS][STAGES];
  __shared__ float ml_s[WARPS][2 * ROWS];
  // the join kernel may be launched now; it waits for this grid's end before it reads
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (p.follows) asm volatile("griddepcontrol.wait;" ::: "memory");   // for the selected lists
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const thin_attn_paged_attention_args& a = p.a;
  const int G = a.Hq / a.H, tiles = (G + ROWS - 1) / ROWS, HT = a.H * tiles;

  // tokens that see nothing: zeros and -inf
  for (int n = blockIdx.x; n < a.N; n += gridDim.x) {
    const Token t = token_of<S::kUnit>(p, n);
    if (!t.live || t.units) continue;
    for (int i = tid; i < a.Hq * a.D; i += kThreads)
      ((T*)a.out)[n * a.out_token + (i / a.D) * a.out_head + i % a.D] = elem_of<T>(0.f);
    if (a.lse)
      for (int i = tid; i < a.Hq; i += kThreads) a.lse[(int64_t)n * a.Hq + i] = -INFINITY;
  }

  // this CTA's stretch [lo, hi) of the line: every thread adds up some tokens, and the threads whose
  // tokens hold lo and hi find the places there
  const int per = (a.N + kThreads - 1) / kThreads;
  const int n0 = min(a.N, tid * per), n1 = min(a.N, n0 + per);
  auto length = [&](int units) { return units ? (int64_t)(units + kPairCost) * HT : 0; };
  int64_t mine = 0;
  for (int n = n0; n < n1; ++n) mine += length(token_of<S::kUnit>(p, n).units);
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) sums[warp] = incl;
  if (tid == 0) parts.cuts[blockIdx.x].n = -1;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) incl += sums[w];
    total += sums[w];
  }
  const int64_t ctas = min(total, (int64_t)gridDim.x);   // no stretch is empty
  if (blockIdx.x >= ctas) return;
  const int64_t lo = total * blockIdx.x / ctas, hi = total * (blockIdx.x + 1) / ctas;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t x = i ? hi - 1 : lo;   // the stretch's first and last place
    if (x < incl - mine || x >= incl) continue;
    int64_t at = incl - mine;
    for (int n = n0;; ++n) {
      const int units = token_of<S::kUnit>(p, n).units;
      if (x < at + length(units)) {
        const int in = (int)((x - at) % (units + kPairCost)) - kPairCost;   // negative: before the pair's units
        ends_s[i] = End{n, (int)((x - at) / (units + kPairCost)), i ? in : max(in, 0)};
        break;
      }
      at += length(units);
    }
  }
  __syncthreads();
  const End end = ends_s[1];   // the last place: unit `unit` of the pair, -1 or less: none of its units

  // the filling side's place: token, head tile, unit of the pair
  int n = ends_s[0].n, tile = ends_s[0].tile, unit = ends_s[0].unit;
  const int first_unit = unit;
  Token tok = token_of<S::kUnit>(p, n);
  int raw_row, raw_len;   // of the token behind it, fetched ahead
  auto peek = [&]() {
    const int next = min(n + 1, a.N - 1);
    raw_row = a.rows ? a.rows[next] : next;
    raw_len = p.keys[next];
  };
  peek();
  // whether the filling side has come to the stretch's end
  auto ended = [&]() { return n > end.n || (n == end.n && (tile > end.tile || (tile == end.tile && unit > end.unit))); };
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * STAGES * S::kStage;
  float4* const merge = (float4*)(smem + S::kRing);
  float* const scratch = (float*)(smem + S::kRing + S::kMerge);
  if (a.E < HD) {
    // the columns behind E are never written again
    for (int i = lane; i < STAGES * S::kStage / 16; i += 32) *(uint4*)(smem + warp * STAGES * S::kStage + i * 16) = make_uint4(0, 0, 0, 0);
    __syncwarp();
  }
  constexpr int kRun = kKeys < 16 ? kKeys : 16;
  const bool whole = a.page % kRun == 0;   // kRun neighbouring keys of a stage lie on one page
  const int row_key = lane & (kKeys - 1);
  // the filling side's key head
  const C *k_head, *v_head;
  const int32_t* ids;
  auto at_head = [&]() {
    const int h = tile / tiles;
    k_head = (const C*)a.k_pages + h * a.kp_head;
    v_head = (const C*)a.v_pages + h * a.vp_head;
    ids = tok.ids + h * p.ids_head;
  };
  int id = -1, off = 0;
  bool on = false;
  // the page id of this lane's key at the filling side's place
  auto look = [&]() {
    const int key = (tok.start & ~(kAlign - 1)) + unit * S::kUnit + warp * kKeys + row_key;
    on = key >= tok.start && key < tok.len;
    const int j = page_of(p, key);
    off = key - j * a.page;
    id = key < tok.len ? ids[j] : -1;
  };
  constexpr int CH = RB / 16;               // pieces of a stage's row
  constexpr int LPR = CH < 32 ? CH : 32;    // lanes per row
  constexpr int RPI = 32 / LPR;             // rows per instruction
  static_assert(RPI == 1 || RPI == 2 || RPI == 4, "");
  const int r0 = lane / LPR, piece = lane % LPR;
  const int k_pieces = a.E * (int)sizeof(C) / 16, v_pieces = a.D * (int)sizeof(C) / 16;
  const uint32_t lane_at = r0 * RB + ((piece ^ ((r0 & 1) << 2)) << 4);
  int filled = 0;
  bool more = !ended();
  auto fill = [&]() {
    if (more) {
      const int st = filled % STAGES;
      const bool held = id >= 0 && id < a.n_pages;
      const uint32_t seen = __ballot_sync(0xffffffffu, on && held) & kAll;
      const uint32_t ks = ring + st * S::kStage;
      const int64_t page = held ? id : 0;
      if (whole && seen == kAll) {
        // kRun rows of a page at a time, a fixed stride apart
#pragma unroll
        for (int run = 0; run < kKeys; run += kRun) {
          const int64_t pg = kKeys == kRun ? page : (int64_t)__shfl_sync(0xffffffffu, id, run);
          const int row0 = kKeys == kRun ? off - row_key : __shfl_sync(0xffffffffu, off, run);
          const C* kr = k_head + pg * a.kp_page + (row0 + r0) * a.kp_row + piece * (16 / (int)sizeof(C));
          const C* vr = v_head + pg * a.vp_page + (row0 + r0) * a.vp_row + piece * (16 / (int)sizeof(C));
#pragma unroll
          for (int i = 0; i < kRun / RPI; ++i) {
            const int row = run + i * RPI;   // swizzle(row + r0) = swizzle(row) ^ ((r0 & 1) << 2)
            const uint32_t at = ks + row * RB + (lane_at ^ (Tile::swizzle(row) << 4));
#pragma unroll
            for (int x = 0; x < CH; x += LPR) {
              if (piece + x < k_pieces) cp16(at + x * 16, (const char*)kr + x * 16);
              if (piece + x < v_pieces) cp16(at + kKeys * RB + x * 16, (const char*)vr + x * 16);
            }
            kr += RPI * a.kp_row;
            vr += RPI * a.vp_row;
          }
        }
      } else {
        const int64_t ko = page * a.kp_page + off * a.kp_row, vo = page * a.vp_page + off * a.vp_row;
#pragma unroll
        for (int i = 0; i < kKeys / RPI; ++i) {
          const int row = i * RPI + r0;
          const bool full = (seen >> row) & 1;
          const C *kr = k_head + __shfl_sync(0xffffffffu, ko, row), *vr = v_head + __shfl_sync(0xffffffffu, vo, row);
          const uint32_t at = ks + i * RPI * RB + (lane_at ^ (Tile::swizzle(i * RPI) << 4));
#pragma unroll
          for (int x = 0; x < CH; x += LPR) {
            if (piece + x < k_pieces) cp16(at + x * 16, full ? (const char*)kr + (piece + x) * 16 : (const char*)a.k_pages, full);
            if (piece + x < v_pieces)
              cp16(at + kKeys * RB + x * 16, full ? (const char*)vr + (piece + x) * 16 : (const char*)a.v_pages, full);
          }
        }
      }
      Meta me{n, tile | (unit == 0 || filled == 0 ? 1 << 30 : 0), seen, tok.units - 1 - unit};
      ++filled;
      if (++unit == tok.units) {
        unit = 0;
        if (++tile == HT) {
          tile = 0;
          while (++n < a.N) {
            tok = token_from<S::kUnit>(p, n, raw_row, raw_len);
            peek();
            if (tok.units) break;
          }
        }
        at_head();
      }
      more = !ended();
      if (more) look();
      if (me.left == 0 || !more) me.tile |= 1 << 31;
      if (lane == 0) meta[warp][st] = me;
    }
    cp_commit();
  };
  at_head();
  if (more) look();
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) fill();

  Tile t;
  int slot = 0;   // 0: the pair at hand is the one that the stretch begins in, 1: a later one
  auto fetch = [&](const Meta& me) {
    const int h = me.which() / tiles, g0 = (me.which() % tiles) * ROWS;
    if constexpr (Tile::kAhead) t.fetch(p, me.n, h * G + g0, min(ROWS, G - g0), lane);
  };
  __syncwarp();
  if (filled) fetch(meta[warp][0]);
  for (int s = 0; s < filled; ++s) {
    cp_wait<STAGES - 2>();
    __syncwarp();
    fill();   // the stage that the last step emptied
    __syncwarp();
    const int st = s % STAGES;
    const Meta me = meta[warp][st];
    const int h = me.which() / tiles, g0 = (me.which() % tiles) * ROWS, rows = min(ROWS, G - g0);
    if (me.first()) {
      slot = s > 0;
      t.reset(p, me.n, h * G + g0, rows, p.scale_log2e * (a.k_scale ? a.k_scale[h] : 1.f), lane,
              Tile::kSmem ? scratch : (float*)(merge + warp * ROWS * (Tile::COLS / 4)));
    }
    if (s + 1 < filled && meta[warp][(s + 1) % STAGES].first()) fetch(meta[warp][(s + 1) % STAGES]);
    const uint32_t ks = ring + st * S::kStage;
    if (me.seen) t.step(p, ks, ks + kKeys * RB, me.seen, lane, scratch);
    if (!me.last()) continue;

    // the pair's end in this CTA: join the warps, and finish the pair or leave a partial
    const bool begins = slot || first_unit == 0, complete = begins && me.left == 0;
    if (begins && !complete && tid == 0)   // the pair's end on the line, and the CTA whose stretch holds it
      parts.cuts[blockIdx.x] = Cut{me.n, me.which(), (int)(((hi + me.left) * ctas - 1) / total), slot};
    t.finish(ml_s[warp], lane);
    const float vscale = a.v_scale ? a.v_scale[h] : 1.f;
    const int64_t part0 = ((int64_t)blockIdx.x * 2 + slot) * ROWS;
    constexpr int COLS = Tile::COLS;
    for (int part = 0; part * COLS < a.D; ++part) {
      t.put(merge + warp * ROWS * (COLS / 4), part, lane);
      __syncthreads();
      for (int i = tid; i < rows * (COLS / 4); i += kThreads) {
        const int g = i / (COLS / 4), d = i % (COLS / 4);
        float mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) mx = fmaxf(mx, ml_s[w][2 * g]);
        const float ref = mx == -INFINITY ? 0.f : mx;
        float l = 0.f;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
          const float f = ex2(ml_s[w][2 * g] - ref);
          const float4 y = merge[w * ROWS * (COLS / 4) + Tile::place(g, d)];
          l = fmaf(ml_s[w][2 * g + 1], f, l);
          x.x = fmaf(y.x, f, x.x);
          x.y = fmaf(y.y, f, x.y);
          x.z = fmaf(y.z, f, x.z);
          x.w = fmaf(y.w, f, x.w);
        }
        const int col = part * COLS + 4 * d;
        if (complete) {
          const float inv = l == 0.f ? 0.f : vscale / l;
          if (col < a.D) {
            T* out = (T*)a.out + me.n * a.out_token + (h * G + g0 + g) * a.out_head + col;
            out[0] = elem_of<T>(x.x * inv);
            out[1] = elem_of<T>(x.y * inv);
            out[2] = elem_of<T>(x.z * inv);
            out[3] = elem_of<T>(x.w * inv);
          }
          if (part == 0 && d == 0 && a.lse)
            a.lse[(int64_t)me.n * a.Hq + h * G + g0 + g] = l == 0.f ? -INFINITY : (mx + log2f(l)) * 0.6931471805599453f;
        } else {
          if (col < a.D) *(float4*)(parts.o + (part0 + g) * a.D + col) = x;
          if (part == 0 && d == 0) {
            parts.ml[2 * (part0 + g)] = mx;
            parts.ml[2 * (part0 + g) + 1] = l;
          }
        }
      }
      __syncthreads();
    }
  }
}

// Joins the partials of the pair that begins in attention CTA blockIdx.x and is cut: a CTA per query row,
// four warps that take every fourth partial.  Two reads one after the other (cut, partials), 3 us behind
// the attention's end; larger CTAs start later (four rows to a CTA: 0.5 to 1.5 us more).
constexpr int kJoinWarps = 4;

template <typename T>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(PagedAttn p, Parts parts, int ROWS) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const thin_attn_paged_attention_args& a = p.a;
  const Cut cut = parts.cuts[blockIdx.x];
  if (cut.n < 0) return;
  const int G = a.Hq / a.H, tiles = (G + ROWS - 1) / ROWS;
  const int h = cut.tile / tiles, g0 = (cut.tile % tiles) * ROWS;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = blockIdx.y;
  __shared__ float o_s[kJoinWarps][256];
  __shared__ float l_s[kJoinWarps];
  if (g >= G - g0) return;   // the last tile of a head has fewer rows
  const int n = cut.last - (int)blockIdx.x + 1;   // the partials: this CTA's, then slot 0 of those behind it
  auto row_of = [&](int i) { return ((int64_t)(blockIdx.x + i) * 2 + (i ? 0 : cut.slot)) * ROWS + g; };
  float m = -INFINITY, l = 0.f;
  float4 x[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
  // kAhead of this warp's partials at a time, the first ones fetched together with the maxima
  constexpr int kAhead = 4;
  float4 v[kAhead][2];
  float2 ml[kAhead];
  auto fetch = [&](int i0) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int64_t row = row_of(min(i0 + kJoinWarps * u, n - 1));
      ml[u] = *(const float2*)(parts.ml + 2 * row);
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int d = lane * 4 + 128 * y;
        if (d < a.D) v[u][y] = *(const float4*)(parts.o + row * a.D + d);
      }
    }
  };
  fetch(warp);
  for (int i = lane; i < n; i += 32) m = fmaxf(m, parts.ml[2 * row_of(i)]);
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float ref = m == -INFINITY ? 0.f : m;
  for (int i0 = warp; i0 < n; i0 += kJoinWarps * kAhead) {
    if (i0 != warp) fetch(i0);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (i0 + kJoinWarps * u >= n) break;
      const float f = ex2(ml[u].x - ref);
      l = fmaf(ml[u].y, f, l);
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        if (lane * 4 + 128 * y >= a.D) continue;
        x[y].x = fmaf(v[u][y].x, f, x[y].x);
        x[y].y = fmaf(v[u][y].y, f, x[y].y);
        x[y].z = fmaf(v[u][y].z, f, x[y].z);
        x[y].w = fmaf(v[u][y].w, f, x[y].w);
      }
    }
  }
  *(float4*)(o_s[warp] + lane * 4) = x[0];
  *(float4*)(o_s[warp] + 128 + lane * 4) = x[1];
  if (lane == 0) l_s[warp] = l;
  __syncthreads();
  l = (l_s[0] + l_s[1]) + (l_s[2] + l_s[3]);
  const float inv = l == 0.f ? 0.f : (a.v_scale ? a.v_scale[h] : 1.f) / l;
  T* out = (T*)a.out + cut.n * a.out_token + (h * G + g0 + g) * a.out_head;
  for (int d = threadIdx.x; d < a.D; d += kJoinWarps * 32)
    out[d] = elem_of<T>(((o_s[0][d] + o_s[1][d]) + (o_s[2][d] + o_s[3][d])) * inv);
  if (threadIdx.x == 0 && a.lse)
    a.lse[(int64_t)cut.n * a.Hq + h * G + g0 + g] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }

// Query rows of a tile: up to 8 leave its upper half for the operands' lower parts, 9 to 16 fill it (fp32 has
// only the first form); more are several tiles, each a pair of its own on the line that reads the keys again (the 48
// requests above with 16 rows 64 us, with 32 113; as many draft tokens of a request are as many pairs too: four 176).
int rows_of(const thin_attn_paged_attention_args& a) {
  return a.dtype == THIN_ATTN_FP32 || a.Hq / a.H <= 8 ? 8 : 16;
}

struct PartsLayout {
  size_t ml, cuts, bytes;
};
PartsLayout parts_layout(const thin_attn_paged_attention_args& a) {
  const size_t rows = (size_t)kMaxCtas * 2 * rows_of(a);
  PartsLayout l;
  l.ml = al256(rows * a.D * 4);
  l.cuts = l.ml + al256(rows * 8);
  l.bytes = l.cuts + al256(kMaxCtas * sizeof(Cut));
  return l;
}

template <typename Tile, typename T, typename C, int HD, int WARPS, int STAGES, int PER_SM>
cudaError_t launch_tile(const PagedAttn& p, void* ws, cudaStream_t st) {
  using S = Shape<Tile, C, HD, WARPS, STAGES>;
  static_assert((S::kSmem + 2048) * PER_SM <= 228 * 1024, "shared memory: with what the kernel declares and 1 KB of the driver's");
  auto kernel = attention_kernel<Tile, T, C, HD, WARPS, STAGES, PER_SM>;
  static SharedMemory memory;
  cudaError_t e = memory.allow((const void*)kernel, S::kSmem);
  if (e != cudaSuccess) return e;
  const PartsLayout l = parts_layout(p.a);
  Parts parts{(float*)ws, (float*)((char*)ws + l.ml), (Cut*)((char*)ws + l.cuts)};
  // no more CTAs than units that the table can hold
  const int G = p.a.Hq / p.a.H, tiles = (G + Tile::ROWS - 1) / Tile::ROWS;
  const int64_t per_pair = ((int64_t)p.list_width * p.a.page + S::kUnit - 1) / S::kUnit + 1;
  const int64_t most = per_pair * p.a.N * p.a.H * tiles;
  const int grid = (int)(most < 148 * PER_SM ? most : 148 * PER_SM);
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = p.follows ? 1 : 0;
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(WARPS * 32);
  cfg.dynamicSmemBytes = S::kSmem;
  e = cudaLaunchKernelEx(&cfg, kernel, p, parts);
  if (e != cudaSuccess) return e;
  cfg.numAttrs = 1;
  cfg.dynamicSmemBytes = 0;
  cfg.gridDim = dim3(grid, Tile::ROWS < G ? Tile::ROWS : G);
  cfg.blockDim = dim3(kJoinWarps * 32);
  return cudaLaunchKernelEx(&cfg, join_kernel<T>, p, parts, (int)Tile::ROWS);
}

// By the wider of E and D, rounded up to the stage's row; narrower rows are padded in shared memory, not in
// the reads.  Warps, stages and CTAs per SM fill the 227 KB with 64 KB and more of reads in flight per SM.  Rows of up to
// 128 bytes come 32 keys to a stage (the e4m3 requests above in stages of 16 keys: a sixth more time).
template <typename T, int ROWS>
cudaError_t launch_mma(const PagedAttn& p, void* ws, cudaStream_t st) {
  const int w = p.a.E > p.a.D ? p.a.E : p.a.D;
  if (p.a.cache_dtype == THIN_ATTN_E4M3) {
    if (w <= 128) return launch_tile<MmaTile<T, e4m3, 128, ROWS>, T, e4m3, 128, 4, 3, 2>(p, ws, st);
    return launch_tile<MmaTile<T, e4m3, 256, ROWS>, T, e4m3, 256, 4, 3, 2>(p, ws, st);
  }
  if (w <= 64) return launch_tile<MmaTile<T, T, 64, ROWS>, T, T, 64, 4, 3, 2>(p, ws, st);
  if (w <= 128) return launch_tile<MmaTile<T, T, 128, ROWS>, T, T, 128, 4, 3, 2>(p, ws, st);
  return launch_tile<MmaTile<T, T, 256, ROWS>, T, T, 256, 4, 3, 1>(p, ws, st);
}

cudaError_t launch_tf32(const PagedAttn& p, void* ws, cudaStream_t st) {
  const int w = p.a.E > p.a.D ? p.a.E : p.a.D;
  if (w <= 64) return launch_tile<Tf32Tile<64>, float, float, 64, 4, 4, 3>(p, ws, st);
  if (w <= 128) return launch_tile<Tf32Tile<128>, float, float, 128, 4, 3, 2>(p, ws, st);
  return launch_tile<Tf32Tile<256>, float, float, 256, 6, 2, 1>(p, ws, st);
}

}  // namespace

size_t paged_attention_workspace(const thin_attn_paged_attention_args& a) { return parts_layout(a).bytes; }

cudaError_t launch_paged_attention(const PagedAttn& p, void* ws, cudaStream_t st) {
  if (p.a.dtype == THIN_ATTN_FP32) return launch_tf32(p, ws, st);
  const bool few = rows_of(p.a) == 8;
  if (p.a.dtype == THIN_ATTN_BF16) return few ? launch_mma<__nv_bfloat16, 8>(p, ws, st) : launch_mma<__nv_bfloat16, 16>(p, ws, st);
  return few ? launch_mma<__half, 8>(p, ws, st) : launch_mma<__half, 16>(p, ws, st);
}

}  // namespace thin
