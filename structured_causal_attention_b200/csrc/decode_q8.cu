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
// converted codes and the scales stay outside, in fp32:
//   - a query row is multiplied by the power of two that puts its largest
//     magnitude in [2^14, 2^15): exact but for elements 2^29 and more below the
//     largest, which keep an absolute error of 2^-40 of it;
//   - with vs = 2^e * m, 1 <= m < 2, the weight of a key is w_j = 2^(s_j + e_j - M),
//     s in log2 units. M follows the running maximum of s + e: it is set so that
//     the largest weight is 2^13, and again once one passes 2^15, so that w_j m_j
//     fits fp16 (rounding 2^-12, kept down to 2^-27 of the largest weight). The
//     softmax's sum takes the same weights without the scale, l += w_j 2^-e_j, in
//     fp32. So blocks of very different size need no common scale, and O / l
//     needs no correction.
//
// Under INTRA each stream is a problem of its own (g query rows, every n-th
// position), so every loaded key is visible and none is read twice; otherwise
// the n*g rows of a KV head share the keys. A CTA owns (sequence, KV head, stream
// group, 16-row tile, chunk of keys); its warps each stream 32-key tiles of
// their own through a TMA ring of their own, with nothing between warps until
// their states are merged at the end. The kernel writes the output itself where
// one chunk holds the whole cache, else partials that a second kernel joins.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "hd_common.cuh"
#include "launch.h"
#include "tc_ptx.cuh"

namespace hd {

namespace {

constexpr int kQWarps = 4;
constexpr int kQThreads = kQWarps * 32;
constexpr int kQTile = 32;  // keys of a warp's tile
constexpr float kLn2 = 0.69314718055994530942f;

template <int D>
struct Q8Smem {
  static constexpr int KV = kQTile * D;              // bytes of K (or V) of a tile
  static constexpr int STAGES = D == 128 ? 3 : 6;    // ~98 KB a CTA, two CTAs an SM
  static constexpr int RING = kQWarps * STAGES * 2 * KV;
  static constexpr int FAC = kQWarps * kQTile * 16;  // per warp and key: ks, e, 2^-e, m
  static constexpr int MERGE = kQWarps * 16 * (D + 4) * 4;
  static constexpr int BARS = kQWarps * STAGES * 8;
  static constexpr int TOTAL = RING + FAC + BARS + 16 + 1024;  // and the alignment of the ring
  static_assert(MERGE <= RING, "merge buffer");
};

// Offset of 16-byte chunk ch of a row, as TMA's 128-byte (D = 128) or 64-byte
// swizzle places it: the 8 rows that an ldmatrix phase reads fall in different
// banks.
template <int D>
__device__ __forceinline__ uint32_t swz8(int row, int ch) {
  return D == 128 ? row * 128 + ((ch ^ (row & 7)) << 4) : row * 64 + ((ch ^ ((row >> 1) & 3)) << 4);
}

__device__ __forceinline__ void mma_f16_16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

// Row `row` of a stream group: its stream (of the nq), and query head.
struct QRow {
  int s, h;
};
__device__ __forceinline__ QRow q_row(const DecodeQ8Params& p, int grp, int hk, int row) {
  const int g = p.Hq / p.Hkv;
  return {grp * p.spg + row / g, hk * g + row % g};
}

template <int D, int FMT>
__global__ void __launch_bounds__(kQThreads, 2)
    decode_q8_split_kernel(const DecodeQ8Params p, const __grid_constant__ CUtensorMap tmK,
                           const __grid_constant__ CUtensorMap tmV) {
  using SM = Q8Smem<D>;
  constexpr int S = SM::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sRing = smem_u32(smem);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + SM::RING + SM::FAC + SM::BARS);
  long long idx = blockIdx.x;
  const int mt = static_cast<int>(idx % p.mt);
  idx /= p.mt;
  const int split = static_cast<int>(idx % p.splits);
  idx /= p.splits;
  const int grp = static_cast<int>(idx % p.groups);
  idx /= p.groups;
  const int hk = static_cast<int>(idx % p.Hkv);
  const int b = static_cast<int>(idx / p.Hkv);

  const int T1 = p.seqlen[b];
  const bool ok = T1 >= 1 && T1 <= p.Tcap;
  if (!ok && tid == 0 && mt == 0 && split == 0 && grp == 0 && hk == 0) record_status(p.status, HD_ERR_DEVICE_INDEX);
  const int T = ok ? T1 - 1 : 0;
  const bool intra = p.kpt == 1 && p.n > 1;       // keys are the tokens of one stream
  const int kend = ok ? T1 * p.kpt : 0;
  const int pmin = intra ? T : T * p.n + p.s0;    // the first and last query's own key
  const int pmax = intra ? T : T * p.n + p.s0 + p.nq - 1;
  const int kbeg = max(0, pmin - p.win + 1);      // (win is beyond any cache where there is none)
  const int cs = kbeg + split * p.chunk;
  const int ce = min(kend, cs + p.chunk);
  const long long part_row0 = ((static_cast<long long>(b) * p.Hkv + hk) * p.groups + grp) * p.mt * 16 + mt * 16;

  if (cs >= ce) {  // nothing to read in this chunk
    if (tid < 16) {
      if (p.splits > 1) {
        if (in_bounds((part_row0 + tid) * p.splits + split, 1, p.ext_part, p.status)) {
          float* ml = p.part_ml + ((part_row0 + tid) * p.splits + split) * 2;
          ml[0] = -INFINITY;
          ml[1] = 0.f;
        }
      } else if (mt * 16 + tid < p.rows) {  // no sequence at all: a row of zeros
        const QRow r = q_row(p, grp, hk, mt * 16 + tid);
        const long long oi = ((static_cast<long long>(b) * p.nq + r.s) * p.Hq + r.h) * D;
        const long long li = (static_cast<long long>(b) * p.Hq + r.h) * p.nq + r.s;
        if (in_bounds(oi, D, p.ext_q, p.status) && in_bounds(li, 1, p.ext_lse, p.status)) {
          for (int i = 0; i < D; i += 8) *reinterpret_cast<uint4*>(p.o + oi + i) = make_uint4(0, 0, 0, 0);
          p.lse[li] = -INFINITY;
        }
      }
    }
    return;
  }

  // ---- this warp's tiles: warp, warp + 4, ... of the chunk
  const int all_tiles = (ce - cs + kQTile - 1) / kQTile;
  const int tiles = (all_tiles - warp + kQWarps - 1) / kQWarps;
  const uint32_t ring = sRing + warp * S * 2 * SM::KV;
  const uint32_t bars = sRing + SM::RING + SM::FAC + warp * S * 8;
  const int col = intra ? (p.s0 + grp) * p.Hkv + hk : hk;
  auto load = [&](int i) {
    const uint32_t bar = bars + (i % S) * 8, dst = ring + (i % S) * 2 * SM::KV;
    const int row = cs + (i * kQWarps + warp) * kQTile;
    tc::mbar_expect_tx(bar, 2 * SM::KV);  // rows behind the tensor are filled with zeros and counted
    tc::tma_load_4d(dst, &tmK, bar, 0, col, row, b);
    tc::tma_load_4d(dst + SM::KV, &tmV, bar, 0, col, row, b);
  };
  if (tid == 0) *abort_flag = 0;
  if (lane == 0) {
    for (int i = 0; i < S; ++i) tc::mbar_init(bars + i * 8, 1);
    tc::fence_mbar_init();
    tc::fence_async_smem();
    for (int i = 0; i < S && i < tiles; ++i) load(i);
  }
  __syncthreads();

  // ---- the scales: lane i has key i of the tile. Its place (block, token in the
  // block, stream) moves on by kQWarps tiles a step, without a division.
  const long long sc0 = (static_cast<long long>(b) * p.Hkv + hk) * p.nb * p.n;
  int key = cs + warp * kQTile + lane;
  int stream = intra ? p.s0 + grp : key % p.n;
  int tok = intra ? key : key / p.n;
  int blk = tok / p.bt, off = tok - blk * p.bt;
  const int step_stream = intra ? 0 : (kQWarps * kQTile) % p.n;
  const int step_tok = intra ? kQWarps * kQTile : kQWarps * kQTile / p.n;
  const int step_blk = step_tok / p.bt, step_off = step_tok - step_blk * p.bt;
  float ks = 0.f, vs = 1.f;
  auto fetch_scales = [&]() {
    ks = 0.f;
    vs = 1.f;
    const long long si = sc0 + static_cast<long long>(blk) * p.n + stream;
    if (key < ce && in_bounds(si, 1, p.ext_scale, p.status)) {
      ks = __ldg(p.ks + si);
      vs = __ldg(p.vs + si);
    }
    key += kQWarps * kQTile;
    blk += step_blk;
    off += step_off;
    stream += step_stream;
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

  // ---- Q: rows lane/4 and lane/4 + 8 of the tile. A register of an MMA's B
  // operand holds four codes in a row of a key; so the k index 2t, 2t+1, 2t+8,
  // 2t+9 of a step stands for d = 4t .. 4t+3 of its 16.
  int prow[2];
  float rfac[2];  // score factor of the row: scale * log2(e) over the row's power of two
  uint32_t qf[D / 16][4];
#pragma unroll
  for (int hr = 0; hr < 2; ++hr) {
    const int row = mt * 16 + (lane >> 2) + hr * 8;
    const bool valid = row < p.rows;  // other rows are zeros, and are not written
    const QRow qr = q_row(p, grp, hk, valid ? row : 0);
    prow[hr] = intra ? T : T * p.n + p.s0 + qr.s;
    const long long qi = ((static_cast<long long>(b) * p.nq + qr.s) * p.Hq + qr.h) * D;
    const bool inb = in_bounds(qi, D, p.ext_q, p.status);
    uint2 r[D / 16];
    uint32_t am = 0;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      r[kk] = (valid && inb) ? __ldg(reinterpret_cast<const uint2*>(p.q + qi + kk * 16 + (lane & 3) * 4))
                             : make_uint2(0, 0);
      am = __vmaxu2(am, __vmaxu2(r[kk].x & 0x7fff7fffu, r[kk].y & 0x7fff7fffu));
    }
    am = max(am & 0xffffu, am >> 16);
    am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
    am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
    // exponent of the row's largest magnitude; an infinity or NaN stays one
    const int e = max(static_cast<int>(am >> 7), 1) - 127;
    const int up = min(max(14 - e, -126), 126);
    const float f = __int_as_float((up + 127) << 23);
    rfac[hr] = p.scale_log2 * __int_as_float((127 - up) << 23);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      qf[kk][hr] = pack_half(__uint_as_float(r[kk].x << 16) * f, __uint_as_float(r[kk].x & 0xffff0000u) * f);
      qf[kk][2 + hr] = pack_half(__uint_as_float(r[kk].y << 16) * f, __uint_as_float(r[kk].y & 0xffff0000u) * f);
    }
  }
  // o[c][h]: d = c*16 + 4t + h and + 2 + h (h = 0, 1) of rows lane/4, lane/4 + 8
  float o[D / 16][2][4];
#pragma unroll
  for (int c = 0; c < D / 16; ++c)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[c][0][e] = o[c][1][e] = 0.f;
  float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};

  float4* fac = reinterpret_cast<float4*>(smem + SM::RING) + warp * kQTile;
  int done = 0;  // tiles whose copies have arrived
  for (; done < tiles; ++done) {
    const int st = done % S;
    const int base = cs + (done * kQWarps + warp) * kQTile;
    const uint32_t kb = ring + st * 2 * SM::KV, vb = kb + SM::KV;
    __syncwarp();
    {
      const uint32_t vbits = __float_as_uint(vs);
      const int e = static_cast<int>((vbits >> 23) & 0xffu) - 127;
      const bool fin = e < 128 && e > -127;
      // A scale that is no number (its block took in one) makes the scores of its
      // visible keys NaN. One of zero (never written) is the smallest, of zeros.
      fac[lane] = make_float4(ks, e == 128 ? __int_as_float(0x7fffffff) : static_cast<float>(fin ? e : kQ8MinExp),
                              __int_as_float((127 - (fin ? e : (e == 128 ? 0 : kQ8MinExp))) << 23),
                              fin ? __uint_as_float((vbits & 0x007fffffu) | 0x3f800000u) : 0.f);
    }
    fetch_scales();  // of the next tile
    if (!tc::mbar_wait_warp(bars + st * 8, (done / S) & 1, abort_flag, p.status)) break;
    if (base + kQTile > ce) {
      // V rows behind the chunk may hold anything, and zero times a NaN is one
      for (int i = lane; i < kQTile * D / 16; i += 32)
        if (base + i / (D / 16) >= ce)
          asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};\n" ::"r"(vb + swz8<D>(i / (D / 16), i % (D / 16))), "r"(0)
                       : "memory");
    }
    __syncwarp();

    float s[kQTile / 8][4];
#pragma unroll
    for (int j = 0; j < kQTile / 8; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
#pragma unroll
    for (int c4 = 0; c4 < D / 16; c4 += 4)
#pragma unroll
      for (int j = 0; j < kQTile / 8; ++j) {  // 8 keys, 64 of d
        uint32_t r[4];
        ldsm_x4(kb + swz8<D>(j * 8 + (lane & 7), c4 + (lane >> 3)), r[0], r[1], r[2], r[3]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t b0, b1;
          to_half<FMT, true>(r[i], b0, b1);
          mma_f16_16816(s[j], qf[c4 + i], b0, b1);
        }
      }
    float mx[2] = {-INFINITY, -INFINITY};
    const bool all_seen = base + kQTile <= ce && base + kQTile - 1 <= pmin && pmax - base < p.win;
#pragma unroll
    for (int j = 0; j < kQTile / 8; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int k = j * 8 + (lane & 3) * 2 + e;
        const float2 f = *reinterpret_cast<const float2*>(fac + k);
#pragma unroll
        for (int hr = 0; hr < 2; ++hr) {
          float& x = s[j][2 * hr + e];
          x = fmaf(x, f.x * rfac[hr], f.y);
          const int c = base + k;
          if (!all_seen && !(c < ce && c <= prow[hr] && prow[hr] - c < p.win)) x = -INFINITY;
          mx[hr] = fmaxf(mx[hr], x);
        }
      }
    if (__any_sync(0xffffffffu, mx[0] > m_run[0] + 15.f || mx[1] > m_run[1] + 15.f)) {
#pragma unroll
      for (int hr = 0; hr < 2; ++hr) {
        float m = fmaxf(mx[hr], __shfl_xor_sync(0xffffffffu, mx[hr], 1));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
        if (m > m_run[hr] + 15.f) {
          const float alpha = fast_exp2(m_run[hr] - (m - 13.f));
          m_run[hr] = m - 13.f;
          l_run[hr] *= alpha;
#pragma unroll
          for (int c = 0; c < D / 16; ++c)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              o[c][h][2 * hr] *= alpha;
              o[c][h][2 * hr + 1] *= alpha;
            }
        }
      }
    }
    uint32_t a[kQTile / 16][4];
    const float mu[2] = {m_run[0] == -INFINITY ? 0.f : m_run[0], m_run[1] == -INFINITY ? 0.f : m_run[1]};
#pragma unroll
    for (int j = 0; j < kQTile / 8; ++j) {
      const float2 f0 = *reinterpret_cast<const float2*>(&fac[j * 8 + (lane & 3) * 2].z);
      const float2 f1 = *reinterpret_cast<const float2*>(&fac[j * 8 + (lane & 3) * 2 + 1].z);
#pragma unroll
      for (int hr = 0; hr < 2; ++hr) {
        const float w0 = fast_exp2(s[j][2 * hr] - mu[hr]), w1 = fast_exp2(s[j][2 * hr + 1] - mu[hr]);
        l_run[hr] = fmaf(w0, f0.x, l_run[hr]);
        l_run[hr] = fmaf(w1, f1.x, l_run[hr]);
        a[j / 2][2 * (j & 1) + hr] = pack_half(w0 * f0.y, w1 * f1.y);
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
          mma_f16_16816(o[c + i][0], a[k16], e0, e1);
          mma_f16_16816(o[c + i][1], a[k16], o0, o1);
        }
      }
    __syncwarp();  // every lane has read the tile before the next one replaces it
    if (lane == 0 && done + S < tiles) load(done + S);
  }
  // (only after a wait gave up) copies in flight end before the CTA does
  for (int i = done; i < tiles && i < done + S; ++i)
    for (const long long t0 = clock64(); !tc::mbar_try_wait(bars + (i % S) * 8, (i / S) & 1);)
      if (clock64() - t0 > (1LL << 28)) break;
  __syncthreads();

  // ---- merge the warps' states in shared memory: per warp [16][D+4] floats
  float* mbuf = reinterpret_cast<float*>(smem);
  constexpr int RS = D + 4;
#pragma unroll
  for (int hr = 0; hr < 2; ++hr) {
    float l = l_run[hr];
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    float* rowp = mbuf + (warp * 16 + (lane >> 2) + hr * 8) * RS;
    if ((lane & 3) == 0) {
      rowp[D] = m_run[hr];
      rowp[D + 1] = l;
    }
#pragma unroll
    for (int c = 0; c < D / 16; ++c)
      *reinterpret_cast<float4*>(rowp + c * 16 + (lane & 3) * 4) =
          make_float4(o[c][0][2 * hr], o[c][1][2 * hr], o[c][0][2 * hr + 1], o[c][1][2 * hr + 1]);
  }
  __syncthreads();
  if (*abort_flag) return;
  for (int i = tid; i < 16 * D / 4; i += kQThreads) {
    const int lr = i / (D / 4), col4 = (i % (D / 4)) * 4;
    if (mt * 16 + lr >= p.rows) continue;
    float mw[kQWarps], m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kQWarps; ++w) {
      mw[w] = mbuf[(w * 16 + lr) * RS + D];
      m = fmaxf(m, mw[w]);
    }
    const float mref = (m == -INFINITY) ? 0.f : m;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float lt = 0.f;
#pragma unroll
    for (int w = 0; w < kQWarps; ++w) {
      const float f = fast_exp2(mw[w] - mref);
      const float4 x = *reinterpret_cast<const float4*>(mbuf + (w * 16 + lr) * RS + col4);
      acc.x += f * x.x;
      acc.y += f * x.y;
      acc.z += f * x.z;
      acc.w += f * x.w;
      lt += f * mbuf[(w * 16 + lr) * RS + D + 1];
    }
    if (p.splits > 1) {
      const long long pi = (part_row0 + lr) * p.splits + split;
      if (!in_bounds(pi, 1, p.ext_part, p.status)) continue;
      *reinterpret_cast<float4*>(p.part_o + pi * D + col4) = acc;
      if (col4 == 0) *reinterpret_cast<float2*>(p.part_ml + pi * 2) = make_float2(m, lt);
    } else {
      const QRow r = q_row(p, grp, hk, mt * 16 + lr);
      const long long oi = ((static_cast<long long>(b) * p.nq + r.s) * p.Hq + r.h) * D;
      const long long li = (static_cast<long long>(b) * p.Hq + r.h) * p.nq + r.s;
      if (!in_bounds(oi, D, p.ext_q, p.status) || !in_bounds(li, 1, p.ext_lse, p.status)) continue;
      const float inv = 1.f / lt;
      *reinterpret_cast<uint2*>(p.o + oi + col4) =
          make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
      if (col4 == 0) p.lse[li] = (m + __log2f(lt)) * kLn2;
    }
  }
}

// One warp a query row: the chunks' partials joined.
template <int D>
__global__ void decode_q8_combine_kernel(const DecodeQ8Params p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long gi = static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + warp;
  const long long problems = static_cast<long long>(p.B) * p.Hkv * p.groups;
  if (gi >= problems * p.rows) return;
  const int row = static_cast<int>(gi % p.rows);
  const long long prob = gi / p.rows;
  const int grp = static_cast<int>(prob % p.groups);
  const int hk = static_cast<int>((prob / p.groups) % p.Hkv);
  const int b = static_cast<int>(prob / (static_cast<long long>(p.groups) * p.Hkv));
  const QRow r = q_row(p, grp, hk, row);
  const long long prow = prob * p.mt * 16 + row;
  const long long oi = ((static_cast<long long>(b) * p.nq + r.s) * p.Hq + r.h) * D;
  const long long li = (static_cast<long long>(b) * p.Hq + r.h) * p.nq + r.s;
  if (!in_bounds(prow * p.splits, p.splits, p.ext_part, p.status) || !in_bounds(oi, D, p.ext_q, p.status) ||
      !in_bounds(li, 1, p.ext_lse, p.status))
    return;

  float mx = -INFINITY;
  for (int j = lane; j < p.splits; j += 32) mx = fmaxf(mx, p.part_ml[(prow * p.splits + j) * 2]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  const float mu = (mx == -INFINITY) ? 0.f : mx;
  constexpr int PER = D / 32;
  float acc[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) acc[i] = 0.f;
  float lt = 0.f;
  for (int j = 0; j < p.splits; ++j) {
    const float* ml = p.part_ml + (prow * p.splits + j) * 2;
    // a chunk without a visible key has sum 0, and its partial O may never have
    // been written; a sum that is no number is carried on
    if (ml[1] == 0.f) continue;
    const float f = fast_exp2(ml[0] - mu);
    lt += f * ml[1];
    const float* po = p.part_o + (prow * p.splits + j) * D;
#pragma unroll
    for (int i = 0; i < PER; ++i) acc[i] += f * po[lane + 32 * i];
  }
  const float inv = lt == 0.f ? 0.f : 1.f / lt;
  __nv_bfloat16* out = p.o + oi;
#pragma unroll
  for (int i = 0; i < PER; ++i) out[lane + 32 * i] = __float2bfloat16_rn(acc[i] * inv);
  if (lane == 0) p.lse[li] = lt == 0.f ? -INFINITY : (mx + __log2f(lt)) * kLn2;
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  if (!fn) {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(ptr);
  }
  return fn;
}

// The codes as (d, head or (stream, head), row, sequence), a box of one tile.
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
            CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int FMT>
cudaError_t launch_decode_q8_d(const DecodeQ8Params& p, cudaStream_t stream) {
  const bool intra = p.kpt == 1 && p.n > 1;
  const long long J = intra ? static_cast<long long>(p.n) * p.Hkv : p.Hkv;
  const long long R = intra ? p.Tcap : static_cast<long long>(p.Tcap) * p.n;
  CUtensorMap mk, mv;
  if (!make_map<D>(&mk, p.kc, J, R, p.B) || !make_map<D>(&mv, p.vc, J, R, p.B)) return cudaErrorInvalidValue;
  const int smem = Q8Smem<D>::TOTAL;
  cudaError_t e = cudaFuncSetAttribute(decode_q8_split_kernel<D, FMT>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const long long blocks = static_cast<long long>(p.B) * p.Hkv * p.groups * p.splits * p.mt;
  decode_q8_split_kernel<D, FMT><<<static_cast<unsigned>(blocks), kQThreads, smem, stream>>>(p, mk, mv);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.splits == 1) return e;
  const long long rows = static_cast<long long>(p.B) * p.Hkv * p.groups * p.rows;
  decode_q8_combine_kernel<D><<<static_cast<unsigned>((rows + 7) / 8), 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

// Chunks of whole rounds of the warps (128 keys), four waves of two CTAs an SM
// where the cache is long enough for chunks of 512 keys and more.
long long decode_q8_most_splits(long long problems, long long keys, int sms) {
  const long long round = kQWarps * kQTile;
  const long long target = static_cast<long long>(sms) * 2 * 4;
  const long long sp = (target + problems - 1) / problems;
  const long long most = (keys + 4 * round - 1) / (4 * round);
  return sp < most ? sp : most;
}

void decode_q8_plan(long long problems, long long keys, int sms, int* splits, int* chunk) {
  const long long round = kQWarps * kQTile;
  const long long sp = decode_q8_most_splits(problems, keys, sms);
  long long ch = (keys + sp - 1) / sp;
  ch = (ch + round - 1) / round * round;
  *splits = static_cast<int>((keys + ch - 1) / ch);
  *chunk = static_cast<int>(ch);
}

cudaError_t launch_decode_q8(const DecodeQ8Params& p, cudaStream_t stream) {
  const bool e4m3 = p.format == HD_Q8_E4M3;
  if (p.D == 64)
    return e4m3 ? launch_decode_q8_d<64, HD_Q8_E4M3>(p, stream) : launch_decode_q8_d<64, HD_Q8_INT8>(p, stream);
  if (p.D == 128)
    return e4m3 ? launch_decode_q8_d<128, HD_Q8_E4M3>(p, stream) : launch_decode_q8_d<128, HD_Q8_INT8>(p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace hd
