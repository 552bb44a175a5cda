// kv_q8.cu - the 8-bit KV cache: quantising rows as they are written, and
// reading them back as bf16.
//
// Page "微信WeLM提出Hidden Decoding：大模型推理新范式" (tahou.com), section
// "中间流的作用验证": every stream keeps its own KV state. So a scale belongs to
// one block of tokens, one stream and one KV head: what a stream stores never
// depends on another stream's values.
//
//   value = code * scale
//   E4M3: scale = 2^j, the smallest with absmax <= 448 * 2^j. Dividing by it
//         is exact, so the one rounding is the one to e4m3.
//   INT8: scale = absmax / 127 rounded up to 8 significant bits. With x and the
//         scale of 8 significant bits each, x / scale is a tie between two
//         codes exactly or at least 1/1020 away from one, so the code is the
//         same in every arithmetic that is right to 2^-11.
//
// A block whose first token is written starts afresh. A block that was begun
// before has its scale raised, if the new rows need it, and its earlier codes
// are then rounded again; it is never lowered, so nothing is rounded twice
// unless the range grew.
//
// Writing: one warp, or for long blocks a few of a CTA, own one (K or V, sequence,
// block, stream, head): they alone read and write that scale and those codes, so
// no atomics and no order between units. They hold the block's rows in registers
// between finding their largest magnitude and storing their codes, so each row is
// read once; of a block longer than the 128 (D = 128) or 256 that eight warps hold, the
// rows past those are read twice. Rows of neighbouring heads are neighbours in memory and so are their
// warps. Reading: eight codes a thread, four such in flight.
//
// HBM bounds both: 4 x 16385 tokens, 4 streams, 8 heads of 128 (3 bytes an element
// of K and V, 1.61 GB) are written in 262 us in E4M3 (6.1 TB/s, 94% of a copy) and
// 292 in INT8, and read in 255 (6.3 TB/s). The appending of one token is a launch:
// 2.3 us.
#include <cuda_fp8.h>

#include "hd_common.cuh"
#include "launch.h"

namespace hd {

namespace {

constexpr int kKvWarps = 8;

// The scale that values up to the bf16 magnitude `abits` (finite) need.
template <int FMT>
__device__ __forceinline__ float scale_for(uint32_t abits) {
  const uint32_t f = abits << 16;
  if (FMT == HD_Q8_E4M3) {
    // |a| = (1 + m) 2^e and 448 = 1.75 * 2^8
    const int j = static_cast<int>(f >> 23) - 127 - 8 + ((f & 0x7fffffu) > 0x600000u ? 1 : 0);
    return __int_as_float((max(j, kQ8MinExp) + 127) << 23);
  }
  const float q = __fdiv_rn(__uint_as_float(f), 127.f);
  const float up = __uint_as_float((__float_as_uint(q) + 0xffffu) & 0xffff0000u);
  return fmaxf(up, __int_as_float((kQ8MinExp + 127) << 23));
}

// Two bf16 values (one register) over the scale.
__device__ __forceinline__ float2 scaled(uint32_t x, float inv) {
  return make_float2(__uint_as_float(x << 16) * inv, __uint_as_float(x & 0xffff0000u) * inv);
}

// Four bf16 values over the scale, as four codes.
template <int FMT>
__device__ __forceinline__ uint32_t quantise4(uint32_t x0, uint32_t x1, float inv) {
  const float2 f = scaled(x0, inv), g = scaled(x1, inv);
  if (FMT == HD_Q8_E4M3) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(g, __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
  }
  // x * (1/scale) is within 2^-15 of x / scale. Rounding it to a multiple of
  // 2^-12 first (adding and subtracting 1.5 * 2^11) restores an exact tie and
  // moves no other value across one; adding 1.5 * 2^23 then leaves the nearest
  // even integer in the low bits.
  const float c = 1.5f * (1 << 11), d = 1.5f * (1 << 23);
  const uint32_t i0 = __float_as_uint(((f.x + c) - c) + d), i1 = __float_as_uint(((f.y + c) - c) + d);
  const uint32_t i2 = __float_as_uint(((g.x + c) - c) + d), i3 = __float_as_uint(((g.y + c) - c) + d);
  return __byte_perm(__byte_perm(i0, i1, 0x0040), __byte_perm(i2, i3, 0x0040), 0x5410);
}

template <int FMT>
__device__ __forceinline__ float code_value(uint32_t c) {
  if (FMT == HD_Q8_E4M3) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(c), __NV_E4M3);
    return __half2float(__half(h));
  }
  return static_cast<float>(static_cast<int8_t>(c));
}

// The codes in the two low bytes.
template <int FMT>
__device__ __forceinline__ float2 code_pair(uint32_t c) {
  if (FMT == HD_Q8_E4M3)
    return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c & 0xffffu), __NV_E4M3)));
  return make_float2(code_value<FMT>(c & 0xffu), code_value<FMT>((c >> 8) & 0xffu));
}

// Four codes again at a larger scale: rn(code * old / now).
template <int FMT>
__device__ __forceinline__ uint32_t requantise4(uint32_t c, float old, float now) {
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float v = __fdiv_rn(code_value<FMT>((c >> (8 * i)) & 0xffu) * old, now);
    const uint32_t q = FMT == HD_Q8_E4M3 ? __nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3)
                                         : static_cast<uint32_t>(static_cast<int>(rintf(v))) & 0xffu;
    r |= q << (8 * i);
  }
  return r;
}

// A barrier of the `count` warps from warp `first` on.
__device__ __forceinline__ void unit_sync(int first, int count) {
  asm volatile("bar.sync %0, %1;\n" ::"r"(1 + first), "r"(count * 32) : "memory");
}

// The range [t0, t0 + len) of sequence b, or false (and the status word) if it
// does not lie in the cache or is longer than the rows given.
__device__ __forceinline__ bool token_range(const KvQ8Params& p, int b, int& t0, int& len, bool report) {
  t0 = p.token_offset ? p.token_offset[b] : 0;
  len = p.lengths ? p.lengths[b] : p.L;
  if (t0 >= 0 && len >= 0 && len <= p.L && static_cast<long long>(t0) + len <= p.Tcap) return true;
  if (report) record_status(p.status, HD_ERR_DEVICE_INDEX);
  return false;
}

// NP: passes (of 32 * 8 / D rows) that a warp holds in registers; p.wpu warps have
// a unit (blocks of 64 tokens, 2 x 8192 of them: 237 us with one warp that reads
// its rows twice, 85 with four). Blocks longer than eight warps hold are read a
// second time for their codes.
template <int D, int FMT, int NP>
__global__ void __launch_bounds__(kKvWarps * 32, NP == 8 ? 3 : 5) kv_write_q8_kernel(const KvQ8Params p) {
  constexpr int LPR = D / 8;      // lanes of a row, eight elements each
  constexpr int RPP = 32 / LPR;   // rows of a pass
  __shared__ uint32_t largest_of[kKvWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = (lane % LPR) * 8;
  const int unit0 = warp / p.wpu * p.wpu;  // the unit's first warp
  const int sub = (warp - unit0) * RPP + lane / LPR, step = p.wpu * RPP;
  const bool is_v = blockIdx.z != 0;
  const __nv_bfloat16* x = is_v ? p.v : p.k;
  uint8_t* codes = is_v ? p.v_codes : p.k_codes;
  float* scales = is_v ? p.v_scale : p.k_scale;
  const uint32_t unit = (blockIdx.x * kKvWarps + warp) / p.wpu;
  const uint32_t bs = p.div_hkv.div(unit);
  const int hk = static_cast<int>(unit - bs * p.Hkv);
  const int jb = static_cast<int>(p.div_n.div(bs));
  const int s = static_cast<int>(bs) - jb * p.n;
  if (jb >= p.blocks) return;
  for (int b = blockIdx.y; b < p.B; b += gridDim.y) {
    int t0, len;
    if (!token_range(p, b, t0, len, lane == 0 && jb == 0) || len == 0) continue;
    const int blk = static_cast<int>(p.div_bt.div(t0)) + jb;
    const long long first = static_cast<long long>(blk) * p.bt;  // the block's first token
    const int end = static_cast<int>(min(first + p.bt, static_cast<long long>(t0) + len));
    const int lo = static_cast<int>(max(first, static_cast<long long>(t0)));  // new rows: tokens lo .. end-1
    if (lo >= end) continue;
    const long long tstep = static_cast<long long>(p.n) * p.Hkv * D;  // elements of a token
    const long long at = (static_cast<long long>(s) * p.Hkv + hk) * D + col;
    const long long xo = (static_cast<long long>(b) * p.L - t0) * tstep + at;
    const long long co = static_cast<long long>(b) * p.Tcap * tstep + at;
    const long long xstep = step * tstep;  // from one row of a thread to its next
    const long long si = ((static_cast<long long>(b) * p.Hkv + hk) * p.nb + blk) * p.n + s;
    if (!in_bounds(si, 1, p.ext_scale, p.status)) continue;
    auto row = [&](int t, long long o) {
      if (t >= end || !in_bounds(o, 8, p.ext_rows, p.status)) return make_uint4(0, 0, 0, 0);
      return __ldg(reinterpret_cast<const uint4*>(x + o));
    };
    auto largest = [](uint32_t am, const uint4& r) {  // of magnitudes, as two bf16 halves
      const uint32_t u = __vmaxu2(r.x & 0x7fff7fffu, r.y & 0x7fff7fffu);
      const uint32_t v = __vmaxu2(r.z & 0x7fff7fffu, r.w & 0x7fff7fffu);
      return __vmaxu2(am, __vmaxu2(u, v));
    };
    const float old = first < t0 ? scales[si] : 0.f;
    uint4 held[NP];
    uint32_t am = 0;
    const int t1 = lo + sub;
    long long at_x = xo + t1 * tstep;
#pragma unroll
    for (int i = 0; i < NP; ++i, at_x += xstep) held[i] = row(t1 + i * step, at_x);
#pragma unroll
    for (int i = 0; i < NP; ++i) am = largest(am, held[i]);
    for (int t = t1 + NP * step; t < end; t += step) am = largest(am, row(t, xo + t * tstep));
    uint32_t abits = __reduce_max_sync(0xffffffffu, max(am & 0xffffu, am >> 16));
    if (p.wpu > 1) {  // (all warps of a unit take the same branches)
      if (lane == 0) largest_of[warp] = abits;
      unit_sync(unit0, p.wpu);
      abits = __reduce_max_sync(0xffffffffu, lane < p.wpu ? largest_of[unit0 + lane] : 0u);
      unit_sync(unit0, p.wpu);
    }
    const bool finite = abits < 0x7f80u;
    float now = finite ? fmaxf(scale_for<FMT>(abits), old) : __int_as_float(0x7fffffff);
    if (old != old) now = old;
    const bool poison = now != now;
    if (warp == unit0 && lane == 0) scales[si] = now;  // every lane's read of the old one is before the reduction
    if (first < t0 && now > old) {
      for (int t = static_cast<int>(first) + sub; t < lo; t += step) {
        const long long o = co + t * tstep;
        if (!in_bounds(o, 8, p.ext_codes, p.status)) continue;
        uint2* c = reinterpret_cast<uint2*>(codes + o);
        const uint2 was = *c;
        *c = make_uint2(requantise4<FMT>(was.x, old, now), requantise4<FMT>(was.y, old, now));
      }
    }
    const float inv = __fdiv_rn(1.f, now);
    auto store = [&](int t, long long o, const uint4& r) {
      if (t >= end || !in_bounds(o, 8, p.ext_codes, p.status)) return;
      *reinterpret_cast<uint2*>(codes + o) =
          poison ? make_uint2(0, 0) : make_uint2(quantise4<FMT>(r.x, r.y, inv), quantise4<FMT>(r.z, r.w, inv));
    };
    long long at_c = co + t1 * tstep;
#pragma unroll
    for (int i = 0; i < NP; ++i, at_c += xstep) store(t1 + i * step, at_c, held[i]);
    for (int t = t1 + NP * step; t < end; t += step) store(t, co + t * tstep, row(t, xo + t * tstep));
  }
}

template <int D, int FMT>
__global__ void __launch_bounds__(256) kv_read_q8_kernel(const KvQ8Params p) {
  constexpr int CPR = D / 8, PER = 4;
  const bool is_v = blockIdx.z != 0;
  const uint8_t* codes = is_v ? p.v_codes : p.k_codes;
  const float* scales = is_v ? p.v_scale : p.k_scale;
  __nv_bfloat16* out = is_v ? p.v_out : p.k_out;
  const uint32_t tchunks = static_cast<uint32_t>(p.n) * p.Hkv * CPR;  // chunks of a token
  const uint32_t chunks = tchunks * p.L;                             // and of a sequence
  for (int b = blockIdx.y; b < p.B; b += gridDim.y) {
    int t0, len;
    if (!token_range(p, b, t0, len, threadIdx.x == 0 && blockIdx.x == 0)) len = 0;
    uint2 c[PER];
    float sc[PER];
    const uint32_t e0 = blockIdx.x * (256 * PER) + threadIdx.x;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const uint32_t e = e0 + j * 256;
      const uint32_t r = e / CPR;                       // (token, stream, head)
      const uint32_t pos = p.div_hkv.div(r), hk = r - pos * p.Hkv;
      const uint32_t t = p.div_n.div(pos), s = pos - t * p.n;
      c[j] = make_uint2(0, 0);
      sc[j] = 0.f;  // rows behind the sequence are zeros
      if (e < chunks && static_cast<int>(t) < len) {
        const uint32_t tok = t0 + t;
        const long long co = (static_cast<long long>(b) * p.Tcap + t0) * tchunks * 8 + static_cast<long long>(e) * 8;
        const long long si =
            ((static_cast<long long>(b) * p.Hkv + hk) * p.nb + p.div_bt.div(tok)) * p.n + s;
        if (in_bounds(co, 8, p.ext_codes, p.status) && in_bounds(si, 1, p.ext_scale, p.status)) {
          c[j] = __ldg(reinterpret_cast<const uint2*>(codes + co));
          sc[j] = __ldg(scales + si);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const uint32_t e = e0 + j * 256;
      const long long o = static_cast<long long>(b) * chunks * 8 + static_cast<long long>(e) * 8;
      if (e >= chunks || !in_bounds(o, 8, p.ext_rows, p.status)) continue;
      uint32_t r[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t w = (k < 2 ? c[j].x : c[j].y) >> ((k & 1) * 16);
        const float2 f = code_pair<FMT>(w);
        r[k] = pack_bf16(f.x * sc[j], f.y * sc[j]);
      }
      *reinterpret_cast<uint4*>(out + o) = make_uint4(r[0], r[1], r[2], r[3]);
    }
  }
}

dim3 kv_grid(long long x, int B) {
  return dim3(static_cast<unsigned>(x), static_cast<unsigned>(B < 65535 ? B : 65535), 2);
}

template <int D, int FMT>
cudaError_t launch_write_d(KvQ8Params p, cudaStream_t stream) {
  constexpr int RPP = 32 * 8 / D;
  // rows of a block that can be new in one call, eight passes of them a warp
  const int rows = p.bt < p.L ? p.bt : p.L;
  p.wpu = 1;
  while (p.wpu < kKvWarps && rows > p.wpu * 8 * RPP) p.wpu *= 2;
  const long long warps = static_cast<long long>(p.blocks) * p.n * p.Hkv * p.wpu;
  const dim3 grid = kv_grid((warps + kKvWarps - 1) / kKvWarps, p.B);
  if (rows <= 2 * RPP)
    kv_write_q8_kernel<D, FMT, 2><<<grid, kKvWarps * 32, 0, stream>>>(p);
  else if (rows <= 4 * RPP)
    kv_write_q8_kernel<D, FMT, 4><<<grid, kKvWarps * 32, 0, stream>>>(p);
  else
    kv_write_q8_kernel<D, FMT, 8><<<grid, kKvWarps * 32, 0, stream>>>(p);
  return cudaGetLastError();
}

template <int D, int FMT>
cudaError_t launch_read_d(const KvQ8Params& p, cudaStream_t stream) {
  const long long chunks = static_cast<long long>(p.L) * p.n * p.Hkv * (D / 8);
  kv_read_q8_kernel<D, FMT><<<kv_grid((chunks + 1023) / 1024, p.B), 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_write_q8(const KvQ8Params& p, cudaStream_t stream) {
  const bool e4m3 = p.format == HD_Q8_E4M3;
  if (p.D == 64) return e4m3 ? launch_write_d<64, HD_Q8_E4M3>(p, stream) : launch_write_d<64, HD_Q8_INT8>(p, stream);
  if (p.D == 128) return e4m3 ? launch_write_d<128, HD_Q8_E4M3>(p, stream) : launch_write_d<128, HD_Q8_INT8>(p, stream);
  return cudaErrorInvalidValue;
}

cudaError_t launch_kv_read_q8(const KvQ8Params& p, cudaStream_t stream) {
  const bool e4m3 = p.format == HD_Q8_E4M3;
  if (p.D == 64) return e4m3 ? launch_read_d<64, HD_Q8_E4M3>(p, stream) : launch_read_d<64, HD_Q8_INT8>(p, stream);
  if (p.D == 128) return e4m3 ? launch_read_d<128, HD_Q8_E4M3>(p, stream) : launch_read_d<128, HD_Q8_INT8>(p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace hd
