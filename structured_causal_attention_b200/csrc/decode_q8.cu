// decode_q8.cu - one multi-stream decode step against the 8-bit KV cache.
//
// Page "微信WeLM提出Hidden Decoding：大模型推理新范式" (tahou.com): sections
// "实验效果与成本分析" (the n streams of the new token in one parallel step;
// decode is bandwidth-bound at small batch) and "中间流的作用验证" (each stream
// keeps its own KV state). Visibility is that of decode.cu; a key's K and V are
// one byte an element with a scale for its block of tokens, stream and head:
//
//   s_j = scale * ks_j * (q . kc_j),  O = sum_j softmax(s)_j vs_j vc_j
//
// Codes of both formats are exact in fp16, so the products run as fp16 MMAs on
// converted codes, the scales outside in fp32. (The 8-bit MMAs were built and
// measured. One on e4m3 operands is made of an fp16 one here and converts them
// itself, the query's terms too: 196 us became 228. INT8's scores on the s8 MMA,
// with a query of two 8-bit terms, are 2-5% faster, but an error of 2^-16 of a
// row's largest element is too much for its lse.) A query row is multiplied by the
// power of two that puts its largest magnitude in [2^14, 2^15): exact but for
// elements 2^29 and more below it, which keep an error of 2^-39 of it.
//
// With s in log2 units the weight of a key is w_j = vs_j 2^(s_j - M). M follows the
// running maximum of s + log2 vs: it is set so that the largest weight is 2^13,
// and again once one passes 2^15, so that weights fit fp16 (rounding 2^-11, kept
// down to 2^-27 of the largest). The softmax's sum takes the same weights without
// the scale, l += w_j / vs_j, in fp32. So blocks of very different size need no
// common scale, and O / l needs no correction. A weight below fp32's range counts
// as none, though in l it may: a CTA that meets scales 2^76 and more apart goes over
// its piece again in plain fp32 (Q8Again; 13 to 15 ms where the loop takes 0.19).
//
// Under INTRA each stream is a problem of its own (g query rows, every n-th
// position), so every loaded key is visible and none is read twice; otherwise
// the n*g rows of a KV head share the keys. A CTA has a tile of 8, 16 or 32 rows: a
// tile of 8 is the N of the MMAs (half the MMAs and exponentials of 16 rows that
// are half padding: 200 -> 190 us, and with two CTAs an SM 176), 16 are their M,
// and of 32 the codes are converted once for two such M (B8, 8192 tokens, 32 rows:
// 194 -> 141 us). The keys meet few rows, so as tcgen05's M of 64 and more the rows
// would be padding. With keys as M the codes of K could be its operand as they lie,
// with the query as three 8-bit terms; that was not built. P cannot be such terms: the
// many small weights of a long cache add up to more than their floor.
//
// The work is one line of rounds of 128 keys for each KV head: all rounds of the
// first problem (sequence, stream group), then of the next, as the lengths on the
// device have it. As many CTAs as fit the GPU at once each take an equal piece of
// a head's line, whatever the lengths, so a ragged batch keeps every SM busy (the
// ragged final INTRA step: 49 -> 42 us). The heads' CTAs walk their lines side by
// side, as neighbouring heads lie side by side in a row of the cache: with one
// line through all heads in turn, whose rows are then fetched in scattered pieces
// of 128 (64) bytes, a step at D = 128 took 10% longer and at D = 64 30%. Within a
// problem a CTA's warps each stream 32-key tiles of their own through a TMA ring
// of their own, with nothing between warps until their states are merged. A
// problem that one CTA has whole is written by it; of the others each part goes
// to the workspace, and a second kernel joins them.
//
// HBM bounds it, at the power cap's clock with the conversions close behind. Held
// for seconds (in short bursts), 16385 tokens, 32/8 heads of 128: B8, 1.08 GB, 193 us
// E4M3 (196) and 213 INT8 (184), its final-stream step 168 (164) and 183 (165), INTRA
// 178 and 186; B64, 8.6 GB, 1.49 ms E4M3 and 1.66 INT8 (5.2 TB/s; 1.39 ms, 6.2 TB/s, before
// the clock falls), INTRA 1.46 and 1.45.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "hd_common.cuh"
#include "launch.h"
#include "tc_ptx.cuh"
#include "tensor_map.h"

namespace hd {

namespace {

constexpr int kQWarps = 4;
constexpr int kQThreads = kQWarps * 32;
constexpr int kQTile = 32;  // keys of a warp's tile
static_assert(kQWarps * kQTile == kQ8Round, "a round");
constexpr float kLn2 = 0.69314718055994530942f;

// CTAs of an SM. The copies that three keep in flight are more than HBM serves
// best, but a tile of 16 rows has so much to compute that three are faster all the
// same: 64 sequences of 16385 tokens in INT8 took 1574 us with three and 1650 with
// two, 8 in E4M3 191 and 196. With 8 rows two are: three and two took 188 and 164 us for
// 8 sequences' final streams in E4M3, 191 and 178 for their INTRA step (INT8 194 and
// 176), 1606 and 1398 for that of 64 in INT8, 374 and 347 for 64 final INTRA streams; only with
// one KV head are three faster (INTRA, 16 sequences: 78 and 82). At D = 64, with tiles
// of half the bytes, three are (102 and 111 us). Two row tiles need the registers of two.
constexpr int q8_ctas_per_sm(int D, int tile_rows) { return tile_rows == 32 || (tile_rows == 8 && D == 128) ? 2 : 3; }

// TR query rows a CTA: 8, 16 or 32 (two tiles of 16, the codes converted once for
// both).
template <int D, int TR>
struct Q8Smem {
  static constexpr int CTAS = q8_ctas_per_sm(D, TR);
  static constexpr int KV = kQTile * D;              // bytes of K (or V) of a tile
  static constexpr int STAGES = (TR <= 16 ? 2 : 3) * (128 / D);
  static constexpr int RING = kQWarps * STAGES * 2 * KV;
  static constexpr int Q = TR * D * 2;          // the query rows in fp16
  static constexpr int FAC = kQWarps * kQTile * 12;  // per warp and key: score factor, log2 vs, 1/vs
  static constexpr int MERGE = kQWarps * TR * (D + 4) * 4;
  static constexpr int BARS = kQWarps * STAGES * 8;
  static constexpr int TOTAL = RING + Q + FAC + BARS + TR * 4 + 16 + 1024;  // and the alignment of the ring
  static_assert(MERGE <= RING, "merge buffer");
};

// Offset of 16-byte chunk ch of a row, as TMA's 128-byte (D = 128) or 64-byte
// swizzle places it: the 8 rows that an ldmatrix phase reads fall in different
// banks.
template <int D>
__device__ __forceinline__ uint32_t swz8(int row, int ch) {
  return D == 128 ? row * 128 + ((ch ^ (row & 7)) << 4) : row * 64 + ((ch ^ ((row >> 1) & 3)) << 4);
}

template <bool FIRST = false>
__device__ __forceinline__ void mma_f16_16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};\n"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(FIRST ? 0.f : d[0]),
        "f"(FIRST ? 0.f : d[1]), "f"(FIRST ? 0.f : d[2]), "f"(FIRST ? 0.f : d[3]));
}

// The codes in bytes (0, 1) and (2, 3) of r (PAIRS), or (0, 2) and (1, 3), as
// two pairs of fp16 values.
template <int FMT, bool PAIRS>
__device__ __forceinline__ void to_half(uint32_t r, uint32_t& a, uint32_t& b) {
  if (FMT == HD_Q8_E4M3) {
    if (!PAIRS) r = __byte_perm(r, 0, 0x3120);
    asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %2;\n cvt.rn.f16x2.e4m3x2 %0, lo;\n"
        " cvt.rn.f16x2.e4m3x2 %1, hi;\n}\n"
        : "=r"(a), "=r"(b)
        : "r"(r));
    return;
  }
  // byte c + 128 in the low bits of fp16 1024 is 1024 + 128 + c
  r ^= 0x80808080u;
  const __half2 off = __half2half2(__ushort_as_half(0x6480));  // 1152
  uint32_t x = __byte_perm(r, 0x64646464u, PAIRS ? 0x4140 : 0x4240);
  uint32_t y = __byte_perm(r, 0x64646464u, PAIRS ? 0x4342 : 0x4341);
  const __half2 hx = __hsub2(*reinterpret_cast<__half2*>(&x), off), hy = __hsub2(*reinterpret_cast<__half2*>(&y), off);
  a = *reinterpret_cast<const uint32_t*>(&hx);
  b = *reinterpret_cast<const uint32_t*>(&hy);
}

__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint64_t f32x2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t f32x2_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f32x2_add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float2 f32x2_parts(uint64_t a) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(a));
  return f;
}
__device__ __forceinline__ float lds32(uint32_t addr) {
  float r;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(r) : "r"(addr));
  return r;
}
// An 8 x 8 tile of fp16 pairs across the warp, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint64_t lds64(uint32_t addr) {
  uint64_t r;
  asm volatile("ld.shared.b64 %0, [%1];" : "=l"(r) : "r"(addr));
  return r;
}

// Row `row` of a stream group: its stream (of the nq), and query head.
struct QRow {
  int s, h;
};
__device__ __forceinline__ QRow q_row(const DecodeQ8Params& p, int grp, int hk, int row) {
  const int sg = static_cast<int>(p.div_g.div(row));
  return {grp * p.spg + sg, hk * p.g + row - sg * p.g};
}

// Row `row` of group grp of sequence b and KV head hk, among the rows of q and
// out, and its place in lse.
__device__ __forceinline__ long long out_row(const DecodeQ8Params& p, int b, int grp, int hk, int row) {
  const QRow r = q_row(p, grp, hk, row);
  return (static_cast<long long>(b) * p.nq + r.s) * p.Hq + r.h;
}
__device__ __forceinline__ long long lse_at(const DecodeQ8Params& p, int b, int grp, int hk, int row) {
  const QRow r = q_row(p, grp, hk, row);
  return (static_cast<long long>(b) * p.Hq + r.h) * p.nq + r.s;
}
// A sequence whose length is out of range: a row of zeros.
template <int D>
__device__ __forceinline__ void zero_row(const DecodeQ8Params& p, int b, int grp, int hk, int row) {
  const long long o = out_row(p, b, grp, hk, row) * D, li = lse_at(p, b, grp, hk, row);
  if (!in_bounds(o, D, p.ext_q, p.status) || !in_bounds(li, 1, p.ext_lse, p.status)) return;
  for (int i = 0; i < D; i += 8) *reinterpret_cast<uint4*>(p.o + o + i) = make_uint4(0, 0, 0, 0);
  p.lse[li] = -INFINITY;
}
// Row lr of the row tile at row0 of head hk in the workspace, of the part that a
// CTA has of a problem. Its slot is the problem's number plus the CTA's: along the
// line one or the other grows from part to part, so no two share a slot.
__device__ __forceinline__ long long part_row(const DecodeQ8Params& p, int hk, int row0, int slot, int lr) {
  return (static_cast<long long>(row0) * p.Hkv + static_cast<long long>(hk) * p.tile_rows) * p.slots +
         static_cast<long long>(slot) * p.tile_rows + lr;
}

// Rounds of 128 keys that a problem of sequence b has: 0 where its length is out
// of range.
__device__ __forceinline__ int q8_rounds(const DecodeQ8Params& p, int b) {
  const int T1 = __ldg(p.seqlen + b);
  if (T1 < 1 || T1 > p.Tcap) return 0;
  const int first = p.kpt == 1 && p.n > 1 ? T1 - 1 : (T1 - 1) * p.n + p.s0;  // the first query's own key
  return (T1 * p.kpt - max(0, first - p.win + 1) + kQ8Round - 1) / kQ8Round;
}

// The line of all problems' rounds (of one KV head), and the CTAs' pieces of it.
struct Q8Line {
  int total, piece;
  // Rounds before sequence b.
  __device__ __forceinline__ int before(const DecodeQ8Params& p, int lane, int b) const {
    int sum = 0;
    for (int i = lane; i < b; i += 32) sum += q8_rounds(p, i);
    return __reduce_add_sync(0xffffffffu, sum) * p.groups;
  }
  // The sequence that has round pos < total, and pos within its rounds.
  __device__ __forceinline__ int sequence(const DecodeQ8Params& p, int lane, int pos, int& within) const {
    int start = 0;
    for (int i0 = 0;; i0 += 32) {
      const int mine = i0 + lane < p.B ? q8_rounds(p, i0 + lane) * p.groups : 0;
      int sum = mine;  // of the lanes up to this one
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const int x = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += x;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, start + sum > pos);
      if (past != 0) {
        const int l = __ffs(past) - 1;
        within = pos - start - __shfl_sync(0xffffffffu, sum - mine, l);
        return i0 + l;
      }
      start += __shfl_sync(0xffffffffu, sum, 31);
    }
  }
};
__device__ __forceinline__ Q8Line q8_line(const DecodeQ8Params& p, int lane) {
  int sum = 0;
  for (int i = lane; i < p.B; i += 32) sum += q8_rounds(p, i);
  const int total = __reduce_add_sync(0xffffffffu, sum) * p.groups;
  return {total, max((total + p.ctas - 1) / p.ctas, p.least)};
}

// What the queries see of a warp's tile: keys base .. base + 31, those from `end` on
// behind the piece; all: every row sees every one of them.
struct Q8Seen {
  bool all;
  int base, end, win;
  int t0, g, row0, last;  // own key of row r: t0 + min(row0 + r, last) / g (g = 0: t0)
  __device__ __forceinline__ int own(int r) const { return g ? t0 + min(row0 + r, last) / g : t0; }
};

// l + x * 2^d for d <= 0 and w = 2^d, also where that is below fp32's range and the
// product is not: sums of keys whose V scales differ by all that fp32 spans.
__device__ __forceinline__ float add_scaled(float l, float x, float d, float w) {
  if (d > -100.f) return fmaf(w, x, l);
  const float r = fast_exp2(0.5f * d);
  return fmaf(x * r, r, l);
}

// The state of a warp with 16 RT query rows: rows are the M of its MMAs.
template <int D, int FMT, int RT>
struct Q8Rows {
  static constexpr int ROWS = 16 * RT;
  float rf[RT][2];  // the rows' factors: rows lane/4, lane/4 + 8 of each tile
  // o[rt][c][h]: d = c*16 + 4t + h and + 2 + h (h = 0, 1) of those rows
  float o[RT][D / 16][2][4];
  float m_run[RT][2];
  uint64_t l_run[RT][2];  // two partial sums a row

  __device__ __forceinline__ void start(uint32_t, const float* row_fac, float down, int lane) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
      for (int hr = 0; hr < 2; ++hr) rf[rt][hr] = row_fac[rt * 16 + (lane >> 2) + hr * 8] * down;
#pragma unroll
      for (int c = 0; c < D / 16; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[rt][c][0][e] = o[rt][c][1][e] = 0.f;
      m_run[rt][0] = m_run[rt][1] = -INFINITY;
      l_run[rt][0] = l_run[rt][1] = 0;
    }
  }

  // The tile with its K and V at kb and vb, the keys' factors at sFac.
  __device__ __forceinline__ void tile(uint32_t sQ, uint32_t kb, uint32_t vb, uint32_t sFac, const Q8Seen& seen,
                                       int lane) {
    float s[RT][kQTile / 8][4];
#pragma unroll
    for (int c4 = 0; c4 < D / 16; c4 += 4) {
      uint32_t r[kQTile / 8][4];
#pragma unroll
      for (int j = 0; j < kQTile / 8; ++j)  // 8 keys, 64 of d
        ldsm_x4(kb + swz8<D>(j * 8 + (lane & 7), c4 + (lane >> 3)), r[j][0], r[j][1], r[j][2], r[j][3]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t qf[RT][4];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
          ldsm_x4(sQ + swz(rt * 16 + (lane & 15), (c4 + i) * 2 + (lane >> 4), D / 8), qf[rt][0], qf[rt][1], qf[rt][2],
                  qf[rt][3]);
#pragma unroll
        for (int j = 0; j < kQTile / 8; ++j) {
          uint32_t b0, b1;
          to_half<FMT, true>(r[j][i], b0, b1);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            if (c4 + i == 0)
              mma_f16_16816<true>(s[rt][j], qf[rt], b0, b1);
            else
              mma_f16_16816(s[rt][j], qf[rt], b0, b1);
          }
        }
      }
    }
    uint32_t a[RT][kQTile / 16][4];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      float mx[2] = {-INFINITY, -INFINITY};
      const uint64_t rf2[2] = {pack_f32x2(rf[rt][0], rf[rt][0]), pack_f32x2(rf[rt][1], rf[rt][1])};
#pragma unroll
      for (int j = 0; j < kQTile / 8; ++j) {
        const uint32_t at = sFac + (j * 8 + (lane & 3) * 2) * 4;
        const uint64_t f = lds64(at), lv = lds64(at + kQTile * 4);
#pragma unroll
        for (int hr = 0; hr < 2; ++hr) {
          const uint64_t dot = pack_f32x2(s[rt][j][2 * hr], s[rt][j][2 * hr + 1]);
          const float2 x = f32x2_parts(f32x2_fma(f32x2_mul(dot, rf2[hr]), f, lv));
          s[rt][j][2 * hr] = x.x;
          s[rt][j][2 * hr + 1] = x.y;
        }
      }
      if (!seen.all) {
#pragma unroll
        for (int hr = 0; hr < 2; ++hr) {
          const int own = seen.own(rt * 16 + (lane >> 2) + hr * 8);
#pragma unroll
          for (int j = 0; j < kQTile / 8; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int c = seen.base + j * 8 + (lane & 3) * 2 + e;
              if (!(c < seen.end && c <= own && own - c < seen.win)) s[rt][j][2 * hr + e] = -INFINITY;
            }
        }
      }
#pragma unroll
      for (int j = 0; j < kQTile / 8; ++j)
#pragma unroll
        for (int hr = 0; hr < 2; ++hr) mx[hr] = fmaxf(mx[hr], fmaxf(s[rt][j][2 * hr], s[rt][j][2 * hr + 1]));
      if (__any_sync(0xffffffffu, mx[0] > m_run[rt][0] + 15.f || mx[1] > m_run[rt][1] + 15.f)) {
#pragma unroll
        for (int hr = 0; hr < 2; ++hr) {
          float m = fmaxf(mx[hr], __shfl_xor_sync(0xffffffffu, mx[hr], 1));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
          if (m > m_run[rt][hr] + 15.f) {
            const float alpha = fast_exp2(m_run[rt][hr] - (m - 13.f));
            m_run[rt][hr] = m - 13.f;
            const float2 l = f32x2_parts(l_run[rt][hr]);
            l_run[rt][hr] = pack_f32x2(l.x * alpha, l.y * alpha);
#pragma unroll
            for (int c = 0; c < D / 16; ++c)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                o[rt][c][h][2 * hr] *= alpha;
                o[rt][c][h][2 * hr + 1] *= alpha;
              }
          }
        }
      }
#pragma unroll
      for (int hr = 0; hr < 2; ++hr) {
        const float mu = m_run[rt][hr] == -INFINITY ? 0.f : -m_run[rt][hr];
        const uint64_t mu2 = pack_f32x2(mu, mu);
#pragma unroll
        for (int j = 0; j < kQTile / 8; ++j) {
          const uint64_t iv = lds64(sFac + (2 * kQTile + j * 8 + (lane & 3) * 2) * 4);
          const float2 x = f32x2_parts(f32x2_add(pack_f32x2(s[rt][j][2 * hr], s[rt][j][2 * hr + 1]), mu2));
          const float w0 = fast_exp2(x.x), w1 = fast_exp2(x.y);
          l_run[rt][hr] = f32x2_fma(pack_f32x2(w0, w1), iv, l_run[rt][hr]);
          a[rt][j / 2][2 * (j & 1) + hr] = pack_half(w0, w1);
        }
      }
    }
#pragma unroll
    for (int k16 = 0; k16 < kQTile / 16; ++k16)
#pragma unroll
      for (int c = 0; c < D / 16; c += 2) {  // 16 keys, 32 of d
        uint32_t r[4];
        ldsm_x4_t(vb + swz8<D>(k16 * 16 + (lane & 15), c + (lane >> 4)), r[0], r[1], r[2], r[3]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t e0, o0, e1, o1;
          to_half<FMT, false>(r[2 * i], e0, o0);
          to_half<FMT, false>(r[2 * i + 1], e1, o1);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            mma_f16_16816(o[rt][c + i][0], a[rt][k16], e0, e1);
            mma_f16_16816(o[rt][c + i][1], a[rt][k16], o0, o1);
          }
        }
      }
  }

  // This warp's [ROWS][D+4]: values, reference, sum.
  __device__ __forceinline__ void store(float* to, int lane) const {
    constexpr int RS = D + 4;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int hr = 0; hr < 2; ++hr) {
        const float2 lp = f32x2_parts(l_run[rt][hr]);
        float l = lp.x + lp.y;
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        float* rowp = to + (rt * 16 + (lane >> 2) + hr * 8) * RS;
        if ((lane & 3) == 0) {
          rowp[D] = m_run[rt][hr];
          rowp[D + 1] = l;
        }
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
          *reinterpret_cast<float4*>(rowp + c * 16 + (lane & 3) * 4) =
              make_float4(o[rt][c][0][2 * hr], o[rt][c][1][2 * hr], o[rt][c][0][2 * hr + 1], o[rt][c][1][2 * hr + 1]);
      }
  }
};

// The state of a warp with 8 query rows: keys are the M of its MMAs, the rows their
// N, so that none of M = 16 is padding. S^T = K Q^T leaves a lane with the rows 2t,
// 2t+1 of keys; transposed 8 x 8 by 8 x 8 the weights are the operand of
// O^T = V^T P^T.
template <int D, int FMT>
struct Q8Rows8 {
  static constexpr int ROWS = 8;
  uint64_t rf;            // the factors of rows 2t, 2t+1
  uint32_t qb[D / 16][2];
  float o[D / 16][4];     // d = c*16 + 2g of rows 2t, 2t+1; d + 1 of them (g = lane/4)
  float m_run[2];
  uint64_t l_run;         // of rows 2t, 2t+1, over this lane's keys

  __device__ __forceinline__ void start(uint32_t sQ, const float* row_fac, float down, int lane) {
    rf = pack_f32x2(row_fac[(lane & 3) * 2] * down, row_fac[(lane & 3) * 2 + 1] * down);
#pragma unroll
    for (int c = 0; c < D / 16; c += 2)
      ldsm_x4(sQ + swz(lane & 7, c * 2 + (lane >> 3), D / 8), qb[c][0], qb[c][1], qb[c + 1][0], qb[c + 1][1]);
#pragma unroll
    for (int c = 0; c < D / 16; ++c) o[c][0] = o[c][1] = o[c][2] = o[c][3] = 0.f;
    m_run[0] = m_run[1] = -INFINITY;
    l_run = 0;
  }

  __device__ __forceinline__ void tile(uint32_t, uint32_t kb, uint32_t vb, uint32_t sFac, const Q8Seen& seen, int lane) {
    const int g = lane >> 2;
    float s[kQTile / 16][4];  // of key 16i + g: rows 2t, 2t+1; of key 16i + g + 8: the same
#pragma unroll
    for (int c = 0; c < D / 16; c += 2)
#pragma unroll
      for (int i = 0; i < kQTile / 16; ++i) {  // 16 keys, 32 of d
        uint32_t r[4], a[4];
        ldsm_x4(kb + swz8<D>(i * 16 + (lane & 15), c + (lane >> 4)), r[0], r[1], r[2], r[3]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          to_half<FMT, true>(r[2 * j], a[0], a[2]);
          to_half<FMT, true>(r[2 * j + 1], a[1], a[3]);
          if (c + j == 0)
            mma_f16_16816<true>(s[i], a, qb[c + j][0], qb[c + j][1]);
          else
            mma_f16_16816(s[i], a, qb[c + j][0], qb[c + j][1]);
        }
      }
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int i = 0; i < kQTile / 16; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t at = sFac + (i * 16 + h * 8 + g) * 4;
        const float f = lds32(at), lv = lds32(at + kQTile * 4);
        const float2 x = f32x2_parts(
            f32x2_fma(f32x2_mul(pack_f32x2(s[i][2 * h], s[i][2 * h + 1]), rf), pack_f32x2(f, f), pack_f32x2(lv, lv)));
        s[i][2 * h] = x.x;
        s[i][2 * h + 1] = x.y;
      }
    if (!seen.all) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int own = seen.own((lane & 3) * 2 + e);
#pragma unroll
        for (int i = 0; i < kQTile / 16; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int c = seen.base + i * 16 + h * 8 + g;
            if (!(c < seen.end && c <= own && own - c < seen.win)) s[i][2 * h + e] = -INFINITY;
          }
      }
    }
#pragma unroll
    for (int i = 0; i < kQTile / 16; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) mx[e] = fmaxf(mx[e], fmaxf(s[i][e], s[i][2 + e]));
    if (__any_sync(0xffffffffu, mx[0] > m_run[0] + 15.f || mx[1] > m_run[1] + 15.f)) {
      float alpha[2] = {1.f, 1.f};
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float m = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 4));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
        if (m > m_run[e] + 15.f) {
          alpha[e] = fast_exp2(m_run[e] - (m - 13.f));
          m_run[e] = m - 13.f;
        }
      }
      l_run = f32x2_mul(l_run, pack_f32x2(alpha[0], alpha[1]));
#pragma unroll
      for (int c = 0; c < D / 16; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[c][e] *= alpha[e & 1];
    }
    const uint64_t mu = pack_f32x2(m_run[0] == -INFINITY ? 0.f : -m_run[0], m_run[1] == -INFINITY ? 0.f : -m_run[1]);
#pragma unroll
    for (int i = 0; i < kQTile / 16; ++i) {
      uint32_t b[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float iv = lds32(sFac + (2 * kQTile + i * 16 + h * 8 + g) * 4);
        const float2 x = f32x2_parts(f32x2_add(pack_f32x2(s[i][2 * h], s[i][2 * h + 1]), mu));
        const float w0 = fast_exp2(x.x), w1 = fast_exp2(x.y);
        l_run = f32x2_fma(pack_f32x2(w0, w1), pack_f32x2(iv, iv), l_run);
        b[h] = transpose8(pack_half(w0, w1));
      }
#pragma unroll
      for (int c = 0; c < D / 16; c += 2) {  // 16 keys, 32 of d
        uint32_t r[4], a[4];
        ldsm_x4_t(vb + swz8<D>(i * 16 + (lane & 15), c + (lane >> 4)), r[0], r[1], r[2], r[3]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {  // (row g of M is d = 2g, row g + 8 d = 2g + 1)
          to_half<FMT, false>(r[2 * j], a[0], a[1]);
          to_half<FMT, false>(r[2 * j + 1], a[2], a[3]);
          mma_f16_16816(o[c + j], a, b[0], b[1]);
        }
      }
    }
  }

  __device__ __forceinline__ void store(float* to, int lane) const {
    constexpr int RS = D + 4;
    const float2 lp = f32x2_parts(l_run);
    const float part[2] = {lp.x, lp.y};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float l = part[e];
      l += __shfl_xor_sync(0xffffffffu, l, 4);
      l += __shfl_xor_sync(0xffffffffu, l, 8);
      l += __shfl_xor_sync(0xffffffffu, l, 16);
      float* rowp = to + ((lane & 3) * 2 + e) * RS;
      if (lane < 4) {
        rowp[D] = m_run[e];
        rowp[D + 1] = l;
      }
#pragma unroll
      for (int c = 0; c < D / 16; ++c)
        *reinterpret_cast<float2*>(rowp + c * 16 + (lane >> 2) * 2) = make_float2(o[c][e], o[c][2 + e]);
    }
  }
};

template <int D, int FMT, int TR>
struct Q8RowsOf {
  using type = Q8Rows<D, FMT, TR / 16>;
};
template <int D, int FMT>
struct Q8RowsOf<D, FMT, 8> {
  using type = Q8Rows8<D, FMT>;
};

// A CTA's piece: rounds pos .. end-1 of the line, problem after problem; of sequence b,
// group grp of it, the rounds from r0 on, of `rounds`. (The kernel's own loop is the
// same over plain variables: these members took 16-row tiles' last registers.)
struct Q8Walk {
  int pos, end, b, grp, r0, rounds;
  // False where there is nothing (for p.whole: where the sequence's length is out of range).
  __device__ __forceinline__ bool start(const DecodeQ8Params& p, int cta, int lane) {
    if (p.whole) {  // (a problem a CTA)
      b = static_cast<int>(p.div_groups.div(cta));
      grp = cta - b * p.groups;
      pos = r0 = 0;
      end = rounds = q8_rounds(p, b);
      return rounds != 0;
    }
    const Q8Line line = q8_line(p, lane);
    pos = cta * line.piece;
    end = min(pos + line.piece, line.total);
    if (pos >= end) return false;
    b = line.sequence(p, lane, pos, r0);  // r0: rounds of the sequence before pos
    rounds = q8_rounds(p, b);
    grp = r0 / rounds;
    r0 -= grp * rounds;
    return true;
  }
  // The end of this problem's rounds in the piece.
  __device__ __forceinline__ int last() const { return min(rounds, r0 + end - pos); }
  __device__ __forceinline__ bool next(const DecodeQ8Params& p) {
    pos += last() - r0;
    if (pos >= end) return false;
    r0 = 0;
    if (++grp == p.groups) {
      grp = 0;
      do ++b;
      while ((rounds = q8_rounds(p, b)) == 0);  // (one that is left has rounds: pos < end)
    }
    return true;
  }
};

// A piece in plain fp32, a warp a row: a lane has D / 32 of its elements, the keys
// follow one another. With the weights w = 2^(s + log2 vs - m), as above, but the sum
// l formed from the scores themselves: for scales so far apart that w / vs has lost
// keys that count in l. It stands behind the loop over the piece, as inside it took
// registers of the tiles' (139 -> 146 us at 32 rows of 8192 tokens).
template <int D, int FMT, int ROWS>
struct Q8Again {
  static constexpr int E = D / 32;
  // Codes lane*E .. lane*E + E-1 of a row.
  static __device__ __forceinline__ void codes(const uint8_t* row, int lane, float (&x)[4]) {
    const uint32_t r = E == 4 ? __ldg(reinterpret_cast<const uint32_t*>(row) + lane)
                              : __ldg(reinterpret_cast<const uint16_t*>(row) + lane);
    uint32_t h[2];
    to_half<FMT, true>(r, h[0], h[1]);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h[0]));
    const float2 c = __half22float2(*reinterpret_cast<const __half2*>(&h[1]));
    x[0] = a.x, x[1] = a.y, x[2] = c.x, x[3] = c.y;
  }

  static __device__ __noinline__ void run(const DecodeQ8Params& p) {
    uint32_t block, tid;  // (read again, so that nothing is kept for here)
    asm volatile("mov.u32 %0, %%ctaid.x;\n mov.u32 %1, %%tid.x;\n" : "=r"(block), "=r"(tid));
    const uint32_t line_head = p.div_mt.div(block);
    const int row0 = static_cast<int>(block - line_head * p.mt) * ROWS, valid_rows = min(ROWS, p.rows - row0);
    const int cta = static_cast<int>(p.div_hkv.div(line_head)), hk = static_cast<int>(line_head) - cta * p.Hkv;
    const int warp = static_cast<int>(tid >> 5), lane = static_cast<int>(tid & 31);
    Q8Walk at;
    at.start(p, cta, lane);
    do {
      for (int lr = warp; lr < valid_rows; lr += kQWarps) row(p, at, cta, hk, row0, lr, lane);
    } while (at.next(p));
  }

  static __device__ __forceinline__ void row(const DecodeQ8Params& p, const Q8Walk& at, int cta, int hk, int row0, int lr,
                                             int lane) {
    const int b = at.b, grp = at.grp;
    const bool intra = p.kpt == 1 && p.n > 1;
    const int T = __ldg(p.seqlen + b) - 1, t0 = intra ? T : T * p.n + p.s0;
    const int own = t0 + (intra ? 0 : static_cast<int>(p.div_g.div(row0 + lr)));
    const int kbeg = max(0, t0 - p.win + 1);
    const int from = max(kbeg + at.r0 * kQ8Round, own - p.win + 1);
    const int to = min(min((T + 1) * p.kpt, kbeg + at.last() * kQ8Round), own + 1);
    const long long qrow = out_row(p, b, grp, hk, row0 + lr), li = lse_at(p, b, grp, hk, row0 + lr);
    if (!in_bounds(qrow * D, D, p.ext_q, p.status) || !in_bounds(li, 1, p.ext_lse, p.status)) return;
    float q[E], o[E];
    uint32_t am = 0;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      q[i] = __bfloat162float(p.q[qrow * D + lane * E + i]);
      o[i] = 0.f;
      am = max(am, __float_as_uint(fabsf(q[i])));
    }
    am = __reduce_max_sync(0xffffffffu, am);
    const int up = min(14 - (max(static_cast<int>(am >> 23), 1) - 127), 126);  // the row as the loop has it
    const float rf = am >= 0x7f800000u ? __int_as_float(0x7fffffff) : __int_as_float((127 - up) << 23);
#pragma unroll
    for (int i = 0; i < E; ++i) q[i] *= __int_as_float((127 + up) << 23);
    float m = -INFINITY, l = 0.f;  // l times 2^20: see below
    // key c's codes are at c steps, and a lane looks up the scales of one key of 32
    const long long step = static_cast<long long>(intra ? p.n * p.Hkv : p.Hkv) * D;
    const long long base = (static_cast<long long>(b) * p.Tcap * p.n * p.Hkv +
                            (intra ? (p.s0 + grp) * p.Hkv + hk : hk)) * static_cast<long long>(D);
    const uint8_t *kc = p.kc + base, *vc = p.vc + base;
    const long long sc0 = (static_cast<long long>(b) * p.Hkv + hk) * p.nb * p.n;
    constexpr int U = 4;  // keys in flight
    for (int c32 = from; c32 < to; c32 += 32) {
      const int c = min(c32 + lane, to - 1);
      const int tok = intra ? c : static_cast<int>(p.div_n.div(c)), st = intra ? p.s0 + grp : c - tok * p.n;
      const long long si = sc0 + static_cast<long long>(p.div_bt.div(tok)) * p.n + st;
      float f = 0.f, lv = 0.f;
      if (in_bounds(si, 1, p.ext_scale, p.status)) {
        f = __ldg(p.ks + si) * p.scale_log2;
        const float vs = __ldg(p.vs + si);
        lv = vs == 0.f ? static_cast<float>(kQ8MinExp) : log2f(vs);
      }
      for (int u0 = 0; u0 < min(32, to - c32); u0 += U) {
        float s[U], y[U], v[U][4], top = -INFINITY;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const long long at_key = min(c32 + u0 + u, to - 1) * step;
          float x[4], dot = 0.f;
          codes(kc + at_key, lane, x);
          codes(vc + at_key, lane, v[u]);
#pragma unroll
          for (int i = 0; i < E; ++i) dot = fmaf(q[i], x[i], dot);
#pragma unroll
          for (int d = 16; d > 0; d /= 2) dot += __shfl_xor_sync(0xffffffffu, dot, d);
          const float fu = __shfl_sync(0xffffffffu, f, u0 + u);
          // (dot times either factor alone may pass fp32, and the factors' product where dot is 0)
          s[u] = fabsf(rf * fu) < INFINITY ? dot * (rf * fu) : dot * rf * fu;
          y[u] = s[u] + __shfl_sync(0xffffffffu, lv, u0 + u);
          if (c32 + u0 + u >= to) s[u] = y[u] = -INFINITY;
          top = fmaxf(top, y[u]);
        }
        if (top - 13.f > m) {
          const float d = m - (top - 13.f), alpha = fast_exp2(d);
          l = add_scaled(0.f, l, d, alpha);
#pragma unroll
          for (int i = 0; i < E; ++i) o[i] *= alpha;
          m = top - 13.f;
        }
        const float mu = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const float w = fast_exp2(y[u] - mu);
          // s - m is at most 13 - lv <= 73; with the 2^20 a key that is 2^-36 of the one that set m, of a scale of
          // 2^121, is still in fp32's range, and 2^28 of those of the smallest scale are within it
          l += y[u] == y[u] ? fast_exp2(s[u] - mu + 20.f) : y[u];
#pragma unroll
          for (int i = 0; i < E; ++i) o[i] = fmaf(w, v[u][i], o[i]);
        }
      }
    }
    l *= 0x1p-20f;
    if (at.last() - at.r0 == at.rounds) {
      const float inv = 1.f / l;
#pragma unroll
      for (int i = 0; i < E; ++i) p.o[qrow * D + lane * E + i] = __float2bfloat16_rn(o[i] * inv);
      if (lane == 0) p.lse[li] = (m + __log2f(l)) * kLn2;
      return;
    }
    const long long pi = part_row(p, hk, row0, b * p.groups + grp + cta, lr);
    if (!in_bounds(pi, 1, p.ext_part, p.status)) return;
#pragma unroll
    for (int i = 0; i < E; ++i) p.part_o[pi * D + lane * E + i] = o[i];
    if (lane == 0) reinterpret_cast<float2*>(p.part_ml)[pi] = make_float2(m, l);
  }
};

template <int D, int FMT, int TR>
__global__ void __launch_bounds__(kQThreads, Q8Smem<D, TR>::CTAS)
    decode_q8_split_kernel(const __grid_constant__ DecodeQ8Params p, const __grid_constant__ CUtensorMap tmK,
                           const __grid_constant__ CUtensorMap tmV) {
  using SM = Q8Smem<D, TR>;
  constexpr int S = SM::STAGES, ROWS = TR;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sRing = smem_u32(smem), sQ = sRing + SM::RING;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  float* row_fac = reinterpret_cast<float*>(smem + SM::RING + SM::Q + SM::FAC + SM::BARS);  // [ROWS]
  volatile int* abort_flag = reinterpret_cast<volatile int*>(row_fac + ROWS);
  volatile int* again = abort_flag + 1;  // V scales were too far apart
  const uint32_t bars = sQ + SM::Q + SM::FAC + warp * S * 8;
  const uint32_t ring = sRing + warp * S * 2 * SM::KV;
  if (lane == 0) {
    for (int i = 0; i < S; ++i) tc::mbar_init(bars + i * 8, 1);
    tc::fence_mbar_init();
    tc::fence_async_smem();
  }
  if (tid == 0) {
    *abort_flag = *again = 0;
    tc::tma_prefetch_desc(&tmK);
    tc::tma_prefetch_desc(&tmV);
  }
  if (!p.whole) asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  const uint32_t line_head = p.div_mt.div(blockIdx.x);  // row tiles, then heads, side by side
  const int row0 = static_cast<int>(blockIdx.x - line_head * p.mt) * ROWS, valid_rows = min(ROWS, p.rows - row0);
  const int cta = static_cast<int>(p.div_hkv.div(line_head)), hk = static_cast<int>(line_head) - cta * p.Hkv;
  const bool intra = p.kpt == 1 && p.n > 1;       // keys are the tokens of one stream

  // ---- this CTA's piece: rounds pos .. end-1 of the line; of sequence b, group grp
  // of it, r0 of its `rounds`
  int pos, end, b, grp, r0, rounds;
  if (p.whole) {  // (a problem a CTA)
    b = static_cast<int>(p.div_groups.div(cta));
    grp = cta - b * p.groups;
    rounds = q8_rounds(p, b);
    if (rounds == 0) {
      if (grp == 0 && hk == 0 && tid == 0 && row0 == 0) record_status(p.status, HD_ERR_DEVICE_INDEX);
      if (tid < valid_rows) zero_row<D>(p, b, grp, hk, row0 + tid);
      return;
    }
    pos = r0 = 0;
    end = rounds;
  } else {
    const Q8Line line = q8_line(p, lane);
    pos = cta * line.piece;
    end = min(pos + line.piece, line.total);
    if (pos >= end) return;
    b = line.sequence(p, lane, pos, r0);  // r0: rounds of the sequence before pos
    rounds = q8_rounds(p, b);
    grp = r0 / rounds;
    r0 -= grp * rounds;
  }

  int it = 0;  // tiles of this warp so far: a tile's stage and the parity of its barrier
  while (true) {
  const int r1 = min(rounds, r0 + end - pos);
  const int T = __ldg(p.seqlen + b) - 1;
  const int pmin = intra ? T : T * p.n + p.s0;    // the first and last query's own key
  const int pmax = intra ? T : T * p.n + p.s0 + p.nq - 1;
  const int kbeg = max(0, pmin - p.win + 1);      // (win is beyond any cache where there is none)
  const int cs = kbeg + r0 * kQ8Round;
  const int ce = min((T + 1) * p.kpt, kbeg + r1 * kQ8Round);

  // ---- this warp's tiles: warp, warp + 4, ... of the chunk
  const int all_tiles = (ce - cs + kQTile - 1) / kQTile;
  const int tiles = (all_tiles - warp + kQWarps - 1) / kQWarps;
  const int col = intra ? (p.s0 + grp) * p.Hkv + hk : hk;
  auto load = [&](int i) {
    const uint32_t bar = bars + ((it + i) % S) * 8, dst = ring + ((it + i) % S) * 2 * SM::KV;
    const int row = cs + (i * kQWarps + warp) * kQTile;
    tc::mbar_expect_tx(bar, 2 * SM::KV);  // rows behind the tensor are filled with zeros and counted
    tc::tma_load_4d(dst, &tmK, bar, 0, col, row, b);
    tc::tma_load_4d(dst + SM::KV, &tmV, bar, 0, col, row, b);
  };
  if (lane == 0)
    for (int i = 0; i < S && i < tiles; ++i) load(i);

  // ---- the scales: lane i has key i of the tile. Its place (block, token in the
  // block, stream) moves on by kQWarps tiles a step, without a division.
  const long long sc0 = (static_cast<long long>(b) * p.Hkv + hk) * p.nb * p.n;
  int key = cs + warp * kQTile + lane;
  int tok = intra ? key : static_cast<int>(p.div_n.div(key));
  int stream = intra ? p.s0 + grp : key - tok * p.n;
  int blk = static_cast<int>(p.div_bt.div(tok)), off = tok - blk * p.bt;
  float ks, vs;
  auto fetch_scales = [&]() {
    ks = vs = 0.f;  // behind the piece: as never written, and hidden
    const long long si = sc0 + static_cast<long long>(blk) * p.n + stream;
    if (key < ce && in_bounds(si, 1, p.ext_scale, p.status)) {
      ks = __ldg(p.ks + si);
      vs = __ldg(p.vs + si);
    }
    key += kQWarps * kQTile;
    blk += p.step_blk;
    off += p.step_off;
    stream += p.step_stream;
    if (stream >= p.n) {
      stream -= p.n;
      ++off;
    }
    if (off >= p.bt) {
      off -= p.bt;
      ++blk;
    }
  };
  fetch_scales();

  // ---- Q: the rows in shared memory
#pragma unroll
  for (int i = 0; i < ROWS * (D / 4) / kQThreads; ++i) {
    const int lr = (tid + i * kQThreads) / (D / 4), d4 = (tid + i * kQThreads) % (D / 4);
    uint2 r = make_uint2(0, 0);  // rows past the last are zeros, and are not written
    if (lr < valid_rows) {
      const QRow qr = q_row(p, grp, hk, row0 + lr);
      const long long qi = ((static_cast<long long>(b) * p.nq + qr.s) * p.Hq + qr.h) * D + d4 * 4;
      if (in_bounds(qi, 4, p.ext_q, p.status)) r = __ldg(reinterpret_cast<const uint2*>(p.q + qi));
    }
    uint32_t am = __vmaxu2(r.x & 0x7fff7fffu, r.y & 0x7fff7fffu);
    am = __reduce_max_sync(D == 128 ? 0xffffffffu : 0xffffu << (lane & 16), max(am & 0xffffu, am >> 16));
    const float x[4] = {__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u), __uint_as_float(r.y << 16),
                        __uint_as_float(r.y & 0xffff0000u)};
    const int up = min(14 - (max(static_cast<int>(am >> 7), 1) - 127), 126);
    const float f = __int_as_float((up + 127) << 23);
    // A register of an MMA's B operand holds four codes in a row of a key; so of
    // the 16 k indexes of a step 2t, 2t+1, 2t+8, 2t+9 stand for d = 4t .. 4t+3.
    const uint32_t at = sQ + (d4 & 3) * 4;
    asm volatile("st.shared.b32 [%0], %1;\n" ::"r"(at + swz(lr, (d4 >> 2) * 2, D / 8)), "r"(pack_half(x[0] * f, x[1] * f))
                 : "memory");
    asm volatile("st.shared.b32 [%0], %1;\n" ::"r"(at + swz(lr, (d4 >> 2) * 2 + 1, D / 8)),
                 "r"(pack_half(x[2] * f, x[3] * f))
                 : "memory");
    // (an infinity or NaN in the row: so is every score of it)
    const float fac = am >= 0x7f80u ? __int_as_float(0x7fffffff) : __int_as_float((127 - up) << 23);
    if (d4 == 0) row_fac[lr] = fac;
  }
  __syncthreads();
  typename Q8RowsOf<D, FMT, TR>::type rows;
  // A score is dot * (row's factor) * (key's), from the left, and |dot| < 2^31 (2^15 * 448 * 128). So that no finite
  // row's product with a code passes fp32 where the score does not, a factor of 2^95 and more (a row of 2^109) is
  // taken down to 2^95, all rows' by as much, and the keys' factors up. Those then stop at the largest fp32:
  // scale * scales of 2^110 and more, where that row's scores pass fp32 too or are 0, as they stay.
  const uint32_t rf_bits = lane < ROWS ? __float_as_uint(row_fac[lane]) : 0u;  // (not negative)
  const int rf_top = static_cast<int>(__reduce_max_sync(0xffffffffu, rf_bits < 0x7f800000u ? rf_bits : 0u) >> 23) - 127;
  const int down = max(rf_top - 95, 0);  // at most 18
  rows.start(sQ, row_fac, __int_as_float((127 - down) << 23), lane);
  const float key_fac = p.scale_log2 * __int_as_float((127 + down) << 23);
  const uint32_t sFac = sQ + SM::Q + warp * (kQTile * 12);
  float* fac = reinterpret_cast<float*>(smem + SM::RING + SM::Q) + warp * (kQTile * 3);
  float vs_lo = INFINITY, vs_hi = 0.f;  // V scales of this lane's keys
  int done = 0;  // tiles whose copies have arrived
  for (; done < tiles; ++done) {
    const int st = (it + done) % S;
    const int base = cs + (done * kQWarps + warp) * kQTile;
    const uint32_t kb = ring + st * 2 * SM::KV, vb = kb + SM::KV;
    {
      const uint32_t vbits = __float_as_uint(vs);
      const int e = static_cast<int>((vbits >> 23) & 0xffu) - 127;
      const bool fin = e < 128 && e > -127;
      if (fin) {
        vs_lo = fminf(vs_lo, vs);
        vs_hi = fmaxf(vs_hi, vs);
      }
      // A scale that is no number (its block took in one) makes the scores of its
      // visible keys NaN. One of zero (never written) counts as the smallest.
      const float kf = ks * key_fac;
      fac[lane] = kf == INFINITY ? __int_as_float(0x7f7fffff) : kf;
      fac[kQTile + lane] = fin ? static_cast<float>(e) + __log2f(__uint_as_float((vbits & 0x007fffffu) | 0x3f800000u))
                               : (e == 128 ? __int_as_float(0x7fffffff) : static_cast<float>(kQ8MinExp));
      fac[2 * kQTile + lane] = fin ? __fdividef(1.f, vs) : (e == 128 ? 1.f : __int_as_float((127 - kQ8MinExp) << 23));
    }
    fetch_scales();  // of the next tile
    if (!tc::mbar_wait_warp(bars + st * 8, ((it + done) / S) & 1, abort_flag, p.status)) break;
    if (base + kQTile > ce) {
      // V rows behind the chunk may hold anything, and zero times a NaN is one
      for (int i = lane; i < kQTile * D / 16; i += 32)
        if (base + i / (D / 16) >= ce)
          asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};\n" ::"r"(vb + swz8<D>(i / (D / 16), i % (D / 16))), "r"(0)
                       : "memory");
    }
    __syncwarp();

    const Q8Seen seen = {base + kQTile <= ce && base + kQTile - 1 <= pmin && pmax - base < p.win,
                         base, ce, p.win, intra ? T : T * p.n + p.s0, intra ? 0 : p.g, row0, p.rows - 1};
    rows.tile(sQ, kb, vb, sFac, seen, lane);
    __syncwarp();  // every lane has read the tile and its scales before the next ones replace them
    if (lane == 0 && done + S < tiles) load(done + S);
  }
  // (only after a wait gave up) copies in flight end before the CTA does
  for (int i = done; i < tiles && i < done + S; ++i)
    for (const long long t0 = clock64(); !tc::mbar_try_wait(bars + ((it + i) % S) * 8, ((it + i) / S) & 1);)
      if (clock64() - t0 > (1LL << 28)) break;
  it += tiles;
  __syncthreads();

  // ---- merge the warps' states in shared memory: per warp [ROWS][D+4] floats
  float* mbuf = reinterpret_cast<float*>(smem);
  constexpr int RS = D + 4;
  rows.store(mbuf + warp * ROWS * RS, lane);
  // (columns D + 2 and D + 3 are free; positive floats are ordered as their bits are)
  const uint32_t lo = __reduce_min_sync(0xffffffffu, __float_as_uint(vs_lo));
  const uint32_t hi = __reduce_max_sync(0xffffffffu, __float_as_uint(vs_hi));
  if (lane == 0)
    *reinterpret_cast<uint2*>(mbuf + warp * ROWS * RS + D + 2) = make_uint2(lo, hi);
  __syncthreads();
  if (*abort_flag) return;
  if (tid == 0) {
    float lo4 = INFINITY, hi4 = 0.f;
#pragma unroll
    for (int w = 0; w < kQWarps; ++w) {
      lo4 = fminf(lo4, mbuf[w * ROWS * RS + D + 2]);
      hi4 = fmaxf(hi4, mbuf[w * ROWS * RS + D + 3]);
    }
    // A weight is lost 2^-126 below the reference, 2^-139 of the largest: with scales closer than this its key is
    // 2^-63 of the largest weight's in l.
    if (hi4 * 0x1p-76f > lo4) *again = 1;
  }
  const bool all = r1 - r0 == rounds;
  for (int i = tid; i < valid_rows * (D / 4); i += kQThreads) {
    const int lr = i / (D / 4), col4 = (i % (D / 4)) * 4;
    float mw[kQWarps], m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kQWarps; ++w) {
      mw[w] = mbuf[(w * ROWS + lr) * RS + D];
      m = fmaxf(m, mw[w]);
    }
    const float mref = (m == -INFINITY) ? 0.f : m;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float lt = 0.f;
#pragma unroll
    for (int w = 0; w < kQWarps; ++w) {
      const float f = fast_exp2(mw[w] - mref);
      const float4 x = *reinterpret_cast<const float4*>(mbuf + (w * ROWS + lr) * RS + col4);
      acc.x += f * x.x;
      acc.y += f * x.y;
      acc.z += f * x.z;
      acc.w += f * x.w;
      lt += f * mbuf[(w * ROWS + lr) * RS + D + 1];
    }
    if (all) {
      const long long row = out_row(p, b, grp, hk, row0 + lr), li = lse_at(p, b, grp, hk, row0 + lr);
      if (!in_bounds(row * D, D, p.ext_q, p.status) || !in_bounds(li, 1, p.ext_lse, p.status)) continue;
      const float inv = 1.f / lt;
      *reinterpret_cast<uint2*>(p.o + row * D + col4) =
          make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
      if (col4 == 0) p.lse[li] = (m + __log2f(lt)) * kLn2;
    } else {
      const long long pi = part_row(p, hk, row0, b * p.groups + grp + cta, lr);
      if (!in_bounds(pi, 1, p.ext_part, p.status)) continue;
      *reinterpret_cast<float4*>(p.part_o + pi * D + col4) = acc;
      if (col4 == 0) reinterpret_cast<float2*>(p.part_ml)[pi] = make_float2(m, lt);
    }
  }
  // ---- the next problem of the piece
  pos += r1 - r0;
  if (pos >= end) break;
  r0 = 0;
  if (++grp == p.groups) {
    grp = 0;
    do ++b;
    while ((rounds = q8_rounds(p, b)) == 0);  // (one that is left has rounds: pos < end)
  }
  tc::fence_async_smem();  // the merge's writes come before the copies that replace them
  __syncthreads();
  }
  __syncthreads();
  if (!*again) return;
  Q8Again<D, FMT, ROWS>::run(p);
}

// The parts of a query row joined, one CTA a row: its groups of D / 4 threads
// take the parts in turn, each with a running reference of its own, so that a
// part's reference and values are loaded side by side. Launched while the first
// kernel still runs; what that wrote is there once griddepcontrol.wait returns.
template <int D>
__global__ void __launch_bounds__(kQThreads) decode_q8_combine_kernel(const DecodeQ8Params p) {
  constexpr int LPR = D / 4, G = kQThreads / LPR;
  __shared__ float2 ref[G];
  __shared__ float4 sum[G][LPR];
  const int tid = threadIdx.x, lane = tid & 31;
  const uint32_t unit = p.div_rows.div(blockIdx.x);
  const int row = static_cast<int>(blockIdx.x - unit * p.rows);
  const int prob = static_cast<int>(p.div_hkv.div(unit)), hk = static_cast<int>(unit) - prob * p.Hkv;
  const int b = static_cast<int>(p.div_groups.div(prob)), grp = prob - b * p.groups;
  const int rounds = q8_rounds(p, b);
  const long long orow = out_row(p, b, grp, hk, row), li = lse_at(p, b, grp, hk, row);
  const Q8Line line = q8_line(p, lane);
  const int start = line.before(p, lane, b) + grp * rounds;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  if (rounds == 0) {
    if (tid == 0 && grp == 0 && hk == 0 && row == 0) record_status(p.status, HD_ERR_DEVICE_INDEX);
    if (tid == 0) zero_row<D>(p, b, grp, hk, row);
    return;
  }
  const int cta = start / line.piece, parts = (start + rounds - 1) / line.piece - cta + 1;
  if (parts == 1) return;  // written already
  const int row0 = row / p.tile_rows * p.tile_rows;
  const long long first = part_row(p, hk, row0, prob + cta, row - row0);
  const long long step = p.tile_rows;
  if (!in_bounds(first, (parts - 1) * step + 1, p.ext_part, p.status) || !in_bounds(orow * D, D, p.ext_q, p.status) ||
      !in_bounds(li, 1, p.ext_lse, p.status))
    return;
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int U = 4;  // parts in flight
  for (int j0 = tid / LPR; j0 < parts; j0 += U * G) {
    float2 ml[U];
    float4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // (a part without a key that the row sees has reference -inf, sum 0 and values 0)
      ml[u] = make_float2(-INFINITY, 0.f);
      v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      const long long at = first + (j0 + u * G) * step;
      if (j0 + u * G < parts) {
        ml[u] = reinterpret_cast<const float2*>(p.part_ml)[at];
        v[u] = *reinterpret_cast<const float4*>(p.part_o + at * D + (tid % LPR) * 4);
      }
    }
    float top = m;
#pragma unroll
    for (int u = 0; u < U; ++u) top = fmaxf(top, ml[u].x);
    const float mu = top == -INFINITY ? 0.f : top, f = fast_exp2(m - mu);
    acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float g = fast_exp2(ml[u].x - mu);
      l = u == 0 ? add_scaled(add_scaled(0.f, ml[0].y, ml[0].x - mu, g), l, m - mu, f)
                 : add_scaled(l, ml[u].y, ml[u].x - mu, g);
      acc.x += g * v[u].x;
      acc.y += g * v[u].y;
      acc.z += g * v[u].z;
      acc.w += g * v[u].w;
    }
    m = top;
  }
  if (tid % LPR == 0) ref[tid / LPR] = make_float2(m, l);
  sum[tid / LPR][tid % LPR] = acc;
  __syncthreads();
  if (tid >= LPR) return;
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < G; ++i) top = fmaxf(top, ref[i].x);
  const float mu = top == -INFINITY ? 0.f : top;
  l = 0.f;
  acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < G; ++i) {
    const float g = fast_exp2(ref[i].x - mu);
    const float4 v = sum[i][tid];
    l = add_scaled(l, ref[i].y, ref[i].x - mu, g);
    acc.x += g * v.x;
    acc.y += g * v.y;
    acc.z += g * v.z;
    acc.w += g * v.w;
  }
  const float inv = 1.f / l;
  *reinterpret_cast<uint2*>(p.o + orow * D + tid * 4) =
      make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
  if (tid == 0) p.lse[li] = (top + __log2f(l)) * kLn2;
}

// The codes as (d, head or (stream, head), row, sequence), a box of one tile.
// Promotion to 256 bytes brings the next head's row of a key along: against 128 bytes
// 205 -> 196 us (B8, E4M3, CROSS_FULL), 185 -> 177 under INTRA. Where a row under INTRA has
// fewer than 256 bytes it brings another stream's, used later or not at all: 16 sequences with one
// KV head of 128 take 82 us with it and 68 with 128 bytes, of 64 55 and 51, with two of 64 80 and 74.
template <int D>
bool make_map(CUtensorMap* map, const uint8_t* base, long long J, long long R, long long B) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(J), static_cast<cuuint64_t>(R),
                              static_cast<cuuint64_t>(B)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(J * D),
                                 static_cast<cuuint64_t>(R * J * D)};
  const cuuint32_t box[4] = {D, 1, kQTile, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<uint8_t*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int FMT, int TR>
cudaError_t launch_decode_q8_d(const DecodeQ8Params& p, cudaStream_t stream) {
  const bool intra = p.kpt == 1 && p.n > 1;
  const long long J = intra ? static_cast<long long>(p.n) * p.Hkv : p.Hkv;
  const long long R = intra ? p.Tcap : static_cast<long long>(p.Tcap) * p.n;
  CUtensorMap mk, mv;
  if (!make_map<D>(&mk, p.kc, J, R, p.B) || !make_map<D>(&mv, p.vc, J, R, p.B)) return cudaErrorInvalidValue;
  const int smem = Q8Smem<D, TR>::TOTAL;
  cudaError_t e = cudaFuncSetAttribute(decode_q8_split_kernel<D, FMT, TR>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  decode_q8_split_kernel<D, FMT, TR><<<static_cast<unsigned>(p.ctas * p.Hkv * p.mt), kQThreads, smem, stream>>>(p, mk, mv);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.whole) return e;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.B * p.Hkv * p.groups * p.rows));
  cfg.blockDim = dim3(kQThreads);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode_q8_combine_kernel<D>, p);
}

template <int D, int FMT>
cudaError_t launch_decode_q8_rt(const DecodeQ8Params& p, cudaStream_t stream) {
  if (p.tile_rows == 8) return launch_decode_q8_d<D, FMT, 8>(p, stream);
  if (p.tile_rows == 16) return launch_decode_q8_d<D, FMT, 16>(p, stream);
  if (p.tile_rows == 32) return launch_decode_q8_d<D, FMT, 32>(p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace

// Rows of a CTA.
int decode_q8_tile_rows(int rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : 32; }

// CTAs of a line (of `lines` KV heads and row tiles), the rounds that a piece has at
// least, and whether each CTA takes one problem whole instead of a piece: where
// none has more than kWhole rounds, dividing one and joining its parts takes
// longer than it saves, and the second kernel is left out. It goes by the rounds alone, a
// compromise: in pieces and whole, of 8 rounds, 64 problems and heads (B8 CROSS_FULL) take
// 20.5 and 18.4 us, 256 (INTRA) 26.6 and 22.6, 2048 107 and 89, but 8 16.1 and 18.4; of 16
// rounds 64 26.6 and 26.6, 256 38.9 and 34.8, 2048 185 and 163, but 8 16.4 and 26.6.
void decode_q8_plan(long long problems, long long most_keys, int D, int tile_rows, long long lines, int sms, int* ctas,
                    int* least, int* whole) {
  constexpr int kWhole = 8;
  const long long slots = sms * q8_ctas_per_sm(D, tile_rows) / lines;
  *whole = most_keys <= kWhole * kQ8Round;
  *least = 2;
  *ctas = static_cast<int>(*whole ? problems : (slots > 1 ? slots : 1));
}

cudaError_t launch_decode_q8(const DecodeQ8Params& p, cudaStream_t stream) {
  const bool e4m3 = p.format == HD_Q8_E4M3;
  if (p.D == 64)
    return e4m3 ? launch_decode_q8_rt<64, HD_Q8_E4M3>(p, stream) : launch_decode_q8_rt<64, HD_Q8_INT8>(p, stream);
  if (p.D == 128)
    return e4m3 ? launch_decode_q8_rt<128, HD_Q8_E4M3>(p, stream) : launch_decode_q8_rt<128, HD_Q8_INT8>(p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace hd
