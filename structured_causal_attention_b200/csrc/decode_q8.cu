// decode_q8.cu - one multi-stream decode step against the 8-bit KV cache.
//
// Page "微信WeLM提出Hidden Decoding：大模型推理新范式" (tahou.com): sections
// "实验效果与成本分析" (the n streams of the new token in one parallel step;
// decode is bandwidth-bound at small batch) and "中间流的作用验证" (each stream
// keeps its own KV state). Visibility, query rows and key space are those of
// decode.cu; what differs is that a key's K and V are one byte an element with
// a scale for its block of tokens, stream and head:
//
//   s_j = scale * ks_j * (q . kc_j),  O = sum_j softmax(s)_j vs_j vc_j
//
// Codes of both formats are exact in fp16, so the products run as fp16 MMAs on
// converted codes and the scales stay outside, in fp32:
//   - a query row is multiplied by the power of two that puts its largest
//     magnitude in [2^14, 2^15): exact but for elements 2^29 and more below the
//     largest, which keep an absolute error of 2^-40 of it;
//   - with vs = 2^e * m, 1 <= m < 2, the weight of a key is
//     w_j = 2^(s_j + e_j - M) with M the running maximum of s + e less 14:
//     at most 2^14, so w_j * m_j < 2^15 fits fp16 (rounding 2^-12, kept down to
//     2^-29 of the largest weight). The softmax's sum takes the same weights
//     without the scale, l += w_j * 2^-e_j, in fp32. So blocks of very
//     different size need no common scale, and O / l needs no correction.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "hd_common.cuh"
#include "launch.h"

namespace hd {

namespace {

constexpr int kQWarps = 4;
constexpr int kQThreads = kQWarps * 32;
constexpr int kQBlk = 64;  // keys per stage, 16 a warp
constexpr int kQStages = 4;
constexpr float kLn2 = 0.69314718055994530942f;

template <int D>
struct Q8Smem {
  static constexpr int RC = D / 16;                   // 16-byte chunks of a row of codes
  static constexpr int KV = kQBlk * D;                // bytes of K (or V) of a stage
  static constexpr int STAGE = 2 * KV + 2 * kQBlk * 4;  // and the raw scales of its keys
  static constexpr int FAC = kQWarps * 16 * 16;       // per warp and key: score factor, e, 2^-e, m
  static constexpr int RING = kQStages * STAGE;
  static constexpr int MERGE = kQWarps * 16 * (D + 4) * 4;
  static constexpr int TOTAL = FAC + (RING > MERGE ? RING : MERGE);
};

// Offset of 16-byte chunk ch of a row: chunks of the 8 rows that an ldmatrix
// phase reads fall in different banks (rows of 128 bytes, or two of 64 a line).
template <int D>
__device__ __forceinline__ uint32_t swz8(int row, int ch) {
  return D == 128 ? row * 128 + ((ch ^ (row & 7)) << 4) : row * 64 + ((ch ^ ((row >> 1) & 3)) << 4);
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"(dst), "l"(src));
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
    const __half2_raw x = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(r & 0xffffu), __NV_E4M3);
    const __half2_raw y = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(r >> 16), __NV_E4M3);
    a = x.x | (static_cast<uint32_t>(x.y) << 16);
    b = y.x | (static_cast<uint32_t>(y.y) << 16);
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

template <int D, int FMT>
__global__ void __launch_bounds__(kQThreads, 2) decode_q8_split_kernel(const DecodeQ8Params p) {
  using SM = Q8Smem<D>;
  constexpr int RC = SM::RC;
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t sFac = smem_u32(smem);
  const uint32_t sStage = sFac + SM::FAC;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  long long idx = blockIdx.x;
  const int mt = static_cast<int>(idx % p.mt);
  idx /= p.mt;
  const int split = static_cast<int>(idx % p.splits);
  idx /= p.splits;
  const int hk = static_cast<int>(idx % p.Hkv);
  const int b = static_cast<int>(idx / p.Hkv);
  const int g = p.Hq / p.Hkv;
  const int rows_pad = p.mt * 16;

  const int T1 = p.seqlen[b];
  const bool ok = T1 >= 1 && T1 <= p.Tcap;
  if (!ok && tid == 0 && mt == 0 && split == 0 && hk == 0) record_status(p.status, HD_ERR_DEVICE_INDEX);
  const int T = ok ? T1 - 1 : 0;
  const int kend = ok ? T1 * p.kpt : 0;
  const int kbeg = (p.mode == HD_CROSS_WINDOW) ? max(0, T * p.n + p.s0 - p.win + 1) : 0;
  const int cs = kbeg + split * p.chunk;
  const int ce = min(kend, cs + p.chunk);
  const long long part_row0 = (static_cast<long long>(b) * p.Hkv + hk) * rows_pad + mt * 16;

  if (cs >= ce) {  // nothing to read in this chunk
    if (tid < 16 && in_bounds((part_row0 + tid) * p.splits + split, 1, p.ext_part, p.status)) {
      float* ml = p.part_ml + ((part_row0 + tid) * p.splits + split) * 2;
      ml[0] = -INFINITY;
      ml[1] = 0.f;
    }
    return;
  }

  const long long kv_rs = static_cast<long long>(p.Hkv) * D;
  const long long kv0 = (static_cast<long long>(b) * p.Tcap * p.n * p.Hkv + hk) * D;
  const long long sc0 = (static_cast<long long>(b) * p.Hkv + hk) * p.nb * p.n;
  const int nblk = (ce - cs + kQBlk - 1) / kQBlk;
  auto load_blk = [&](int bi, int st) {
    const int base = cs + bi * kQBlk;
    const uint32_t dk = sStage + st * SM::STAGE, dv = dk + SM::KV;
    for (int i = tid; i < kQBlk * RC; i += kQThreads) {
      const int row = i / RC, ch = i % RC, c = base + row;
      const long long pos = p.kres + static_cast<long long>(min(c, ce - 1)) * p.kstride;
      const long long off = kv0 + pos * kv_rs + ch * 16;
      const bool inb = in_bounds(off, 16, p.ext_cache, p.status);
      const int nb = (c < ce && inb) ? 16 : 0;  // rows behind the chunk are zeros
      cp_async16(dk + swz8<D>(row, ch), p.kc + (inb ? off : 0), nb);
      cp_async16(dv + swz8<D>(row, ch), p.vc + (inb ? off : 0), nb);
    }
    // the scale of a key: K's by the first 64 threads, V's by the others
    const int key = tid % kQBlk;
    const int pos = p.kres + min(base + key, ce - 1) * p.kstride;
    const int tok = pos / p.n;
    const long long si = sc0 + static_cast<long long>(tok / p.bt) * p.n + (pos - tok * p.n);
    const bool inb = in_bounds(si, 1, p.ext_scale, p.status);
    cp_async4(dk + 2 * SM::KV + tid * 4, (tid < kQBlk ? p.ks : p.vs) + (inb ? si : 0));
  };
  static_assert(kQThreads == 2 * kQBlk, "one scale a thread");
#pragma unroll
  for (int i = 0; i < kQStages - 1; ++i) {
    if (i < nblk) load_blk(i, i);
    cp_async_commit();
  }

  // ---- Q: rows lane/4 and lane/4 + 8 of the tile (row i = s*g + j -> q[b, s, hk*g + j, :]).
  // A register of an MMA's B operand holds four codes in a row of a key; so the
  // k index 2t, 2t+1, 2t+8, 2t+9 of a step stands for d = 4t .. 4t+3 of its 16.
  int prow[2], srow[2];
  bool rvalid[2];
  float rfac[2];  // score factor of the row: scale * log2(e) over the row's power of two
  uint32_t qf[D / 16][4];
#pragma unroll
  for (int hr = 0; hr < 2; ++hr) {
    const int row = mt * 16 + (lane >> 2) + hr * 8;
    rvalid[hr] = row < p.rows;
    const int s = rvalid[hr] ? row / g : 0, j = rvalid[hr] ? row % g : 0;
    srow[hr] = p.s0 + s;
    // the query's own key index: its position, or (final stream alone) its token
    prow[hr] = (p.kstride == 1) ? T * p.n + srow[hr] : T;
    const long long qi = ((static_cast<long long>(b) * p.nq + s) * p.Hq + hk * g + j) * D;
    const bool inb = in_bounds(qi, D, p.ext_q, p.status);
    uint2 r[D / 16];
    uint32_t am = 0;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      r[kk] = (rvalid[hr] && inb) ? __ldg(reinterpret_cast<const uint2*>(p.q + qi + kk * 16 + (lane & 3) * 4))
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
  // INTRA: key c is visible iff c % n == s; the offsets' residues are fixed
  int om[2][2];
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int e = 0; e < 2; ++e) om[j][e] = (warp * 16 + j * 8 + (lane & 3) * 2 + e) % p.n;
  // o[c][h]: d = c*16 + 4t + h and + 2 + h (h = 0, 1) of rows lane/4, lane/4 + 8
  float o[D / 16][2][4];
#pragma unroll
  for (int c = 0; c < D / 16; ++c)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[c][0][e] = o[c][1][e] = 0.f;
  float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};

  for (int bi = 0; bi < nblk; ++bi) {
    const int st = bi % kQStages;
    cp_async_wait<kQStages - 2>();
    __syncthreads();
    if (bi + kQStages - 1 < nblk) load_blk(bi + kQStages - 1, (bi + kQStages - 1) % kQStages);
    cp_async_commit();
    const uint32_t kb = sStage + st * SM::STAGE, vb = kb + SM::KV;
    float4* fac = reinterpret_cast<float4*>(smem) + warp * 16;
    if (lane < 16) {
      const float* sc = reinterpret_cast<const float*>(smem + SM::FAC + st * SM::STAGE + 2 * SM::KV) + warp * 16 + lane;
      const float ks = sc[0], vs = sc[kQBlk];
      const uint32_t vbits = __float_as_uint(vs);
      const int e = static_cast<int>((vbits >> 23) & 0xffu) - 127;
      const bool fin = e < 128 && e > -127;
      // A scale that is no number (its block took in one) makes the scores of its
      // visible keys NaN. One of zero (never written) is the smallest, of zeros.
      fac[lane] = make_float4(ks, e == 128 ? __int_as_float(0x7fffffff) : static_cast<float>(fin ? e : kQ8MinExp),
                              __int_as_float((127 - (fin ? e : (e == 128 ? 0 : kQ8MinExp))) << 23),
                              fin ? __uint_as_float((vbits & 0x007fffffu) | 0x3f800000u) : 0.f);
    }
    __syncwarp();
    float s[2][4];
#pragma unroll
    for (int j = 0; j < 2; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int c4 = 0; c4 < RC; c4 += 4) {  // 8 keys, 64 of d
        uint32_t r[4];
        ldsm_x4(kb + swz8<D>(warp * 16 + j * 8 + (lane & 7), c4 + (lane >> 3)), r[0], r[1], r[2], r[3]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t b0, b1;
          to_half<FMT, true>(r[i], b0, b1);
          mma_f16_16816(s[j], qf[c4 + i], b0, b1);
        }
      }
    const int cbase = cs + bi * kQBlk + warp * 16;
    const int bres = (p.mode == HD_INTRA) ? (cs + bi * kQBlk) % p.n : 0;
    float iv[2][2], mant[2][2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int key = j * 8 + (lane & 3) * 2 + e;
        const float4 f = fac[key];
        iv[j][e] = f.z;
        mant[j][e] = f.w;
        const int c = cbase + key;
        int res = 0;
        if (p.mode == HD_INTRA) {
          res = bres + om[j][e];
          res -= (res >= p.n) ? p.n : 0;
        }
#pragma unroll
        for (int hr = 0; hr < 2; ++hr) {
          bool vis = rvalid[hr] && c < ce && c <= prow[hr];
          if (p.mode == HD_INTRA) vis = vis && (res == srow[hr]);
          if (p.mode == HD_CROSS_WINDOW) vis = vis && (prow[hr] - c < p.win);
          float& x = s[j][2 * hr + e];
          x = vis ? fmaf(x, f.x * rfac[hr], f.y) : -INFINITY;
        }
      }
    uint32_t a[4];
#pragma unroll
    for (int hr = 0; hr < 2; ++hr) {
      float mx = fmaxf(fmaxf(s[0][2 * hr], s[0][2 * hr + 1]), fmaxf(s[1][2 * hr], s[1][2 * hr + 1]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float m_new = fmaxf(m_run[hr], mx - 14.f);
      const float m_use = (m_new == -INFINITY) ? 0.f : m_new;
      const float alpha = fast_exp2(m_run[hr] - m_use);
      m_run[hr] = m_new;
      float rs = 0.f;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float w0 = fast_exp2(s[j][2 * hr] - m_use), w1 = fast_exp2(s[j][2 * hr + 1] - m_use);
        rs = fmaf(w0, iv[j][0], rs);
        rs = fmaf(w1, iv[j][1], rs);
        a[2 * j + hr] = pack_half(w0 * mant[j][0], w1 * mant[j][1]);
      }
      l_run[hr] = l_run[hr] * alpha + rs;
#pragma unroll
      for (int c = 0; c < D / 16; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          o[c][h][2 * hr] *= alpha;
          o[c][h][2 * hr + 1] *= alpha;
        }
    }
#pragma unroll
    for (int c = 0; c < D / 16; c += 2) {  // 16 keys, 32 of d
      uint32_t r[4];
      ldsm_x4_t(vb + swz8<D>(warp * 16 + (lane & 15), c + (lane >> 4)), r[0], r[1], r[2], r[3]);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t e0, o0, e1, o1;
        to_half<FMT, false>(r[2 * i], e0, o0);
        to_half<FMT, false>(r[2 * i + 1], e1, o1);
        mma_f16_16816(o[c + i][0], a, e0, e1);
        mma_f16_16816(o[c + i][1], a, o0, o1);
      }
    }
  }
  cp_async_wait<0>();
  __syncthreads();

  // ---- merge the warps' states in shared memory: per warp [16][D+4] floats
  float* mbuf = reinterpret_cast<float*>(smem + SM::FAC);
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
  for (int i = tid; i < 16 * D; i += kQThreads) {
    const int lr = i / D, col = i % D;
    float mw[kQWarps], mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < kQWarps; ++w) {
      mw[w] = mbuf[(w * 16 + lr) * RS + D];
      mx = fmaxf(mx, mw[w]);
    }
    const float mu = (mx == -INFINITY) ? 0.f : mx;
    float acc = 0.f, lt = 0.f;
#pragma unroll
    for (int w = 0; w < kQWarps; ++w) {
      const float f = fast_exp2(mw[w] - mu);
      acc += f * mbuf[(w * 16 + lr) * RS + col];
      lt += f * mbuf[(w * 16 + lr) * RS + D + 1];
    }
    const long long prow_i = (part_row0 + lr) * p.splits + split;
    if (!in_bounds(prow_i, 1, p.ext_part, p.status)) continue;
    p.part_o[prow_i * D + col] = acc;
    if (col == 0) {
      p.part_ml[prow_i * 2] = mx;
      p.part_ml[prow_i * 2 + 1] = lt;
    }
  }
}

template <int D>
__global__ void decode_q8_combine_kernel(const DecodeQ8Params p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long gi = static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + warp;
  const long long total = static_cast<long long>(p.B) * p.Hkv * p.rows;
  if (gi >= total) return;
  const int row = static_cast<int>(gi % p.rows);
  const int hk = static_cast<int>((gi / p.rows) % p.Hkv);
  const int b = static_cast<int>(gi / (static_cast<long long>(p.rows) * p.Hkv));
  const int g = p.Hq / p.Hkv;
  const int s = row / g, h = hk * g + row % g;  // s local to the nq query streams
  const long long prow = (static_cast<long long>(b) * p.Hkv + hk) * (p.mt * 16) + row;
  const long long oi = ((static_cast<long long>(b) * p.nq + s) * p.Hq + h) * D;
  const long long li = (static_cast<long long>(b) * p.Hq + h) * p.nq + s;
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

template <int D, int FMT>
cudaError_t launch_decode_q8_d(const DecodeQ8Params& p, cudaStream_t stream) {
  const int smem = Q8Smem<D>::TOTAL;
  cudaError_t e = cudaFuncSetAttribute(decode_q8_split_kernel<D, FMT>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const long long blocks = static_cast<long long>(p.B) * p.Hkv * p.splits * p.mt;
  decode_q8_split_kernel<D, FMT><<<static_cast<unsigned>(blocks), kQThreads, smem, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const long long rows = static_cast<long long>(p.B) * p.Hkv * p.rows;
  decode_q8_combine_kernel<D><<<static_cast<unsigned>((rows + 7) / 8), 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decode_q8(const DecodeQ8Params& p, cudaStream_t stream) {
  const bool e4m3 = p.format == HD_Q8_E4M3;
  if (p.D == 64)
    return e4m3 ? launch_decode_q8_d<64, HD_Q8_E4M3>(p, stream) : launch_decode_q8_d<64, HD_Q8_INT8>(p, stream);
  if (p.D == 128)
    return e4m3 ? launch_decode_q8_d<128, HD_Q8_E4M3>(p, stream) : launch_decode_q8_d<128, HD_Q8_INT8>(p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace hd
