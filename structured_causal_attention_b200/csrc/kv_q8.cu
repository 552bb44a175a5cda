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
// One warp owns one (K or V, sequence, block, stream, head): it alone reads
// and writes that scale and those codes, so no atomics and no order between
// warps. Rows of neighbouring heads are neighbours in memory and so are their
// warps.
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

// Four bf16 values (two registers) over the scale, as four codes.
template <int FMT>
__device__ __forceinline__ uint32_t quantise4(uint2 x, float inv) {
  const float f0 = __uint_as_float(x.x << 16) * inv, f1 = __uint_as_float(x.x & 0xffff0000u) * inv;
  const float f2 = __uint_as_float(x.y << 16) * inv, f3 = __uint_as_float(x.y & 0xffff0000u) * inv;
  if (FMT == HD_Q8_E4M3) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f0, f1), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f2, f3), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
  }
  // x * (1/scale) is within 2^-15 of x / scale. Rounding it to a multiple of
  // 2^-12 first (adding and subtracting 1.5 * 2^11) restores an exact tie and
  // moves no other value across one; adding 1.5 * 2^23 then leaves the nearest
  // even integer in the low bits.
  const float c = 1.5f * (1 << 11), d = 1.5f * (1 << 23);
  const uint32_t i0 = __float_as_uint(((f0 + c) - c) + d), i1 = __float_as_uint(((f1 + c) - c) + d);
  const uint32_t i2 = __float_as_uint(((f2 + c) - c) + d), i3 = __float_as_uint(((f3 + c) - c) + d);
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

// The range [t0, t0 + len) of sequence b, or false (and the status word) if it
// does not lie in the cache or is longer than the rows given.
__device__ __forceinline__ bool token_range(const KvQ8Params& p, int b, int& t0, int& len, bool report) {
  t0 = p.token_offset ? p.token_offset[b] : 0;
  len = p.lengths ? p.lengths[b] : p.L;
  if (t0 >= 0 && len >= 0 && len <= p.L && static_cast<long long>(t0) + len <= p.Tcap) return true;
  if (report) record_status(p.status, HD_ERR_DEVICE_INDEX);
  return false;
}

template <int D, int FMT>
__global__ void __launch_bounds__(kKvWarps * 32) kv_write_q8_kernel(const KvQ8Params p) {
  constexpr int LPR = D / 4;      // lanes of a row, four elements each
  constexpr int RPP = 32 / LPR;   // rows of a pass
  const int lane = threadIdx.x & 31, sub = lane / LPR, col = (lane % LPR) * 4;
  const long long warps = static_cast<long long>(gridDim.x) * kKvWarps;
  const long long per_tensor = static_cast<long long>(p.B) * p.blocks * p.n * p.Hkv;
  for (long long u = static_cast<long long>(blockIdx.x) * kKvWarps + (threadIdx.x >> 5); u < 2 * per_tensor;
       u += warps) {
    long long i = u;
    const int hk = static_cast<int>(i % p.Hkv);
    i /= p.Hkv;
    const int s = static_cast<int>(i % p.n);
    i /= p.n;
    const int jb = static_cast<int>(i % p.blocks);
    i /= p.blocks;
    const int b = static_cast<int>(i % p.B);
    const bool is_v = i >= p.B;
    int t0, len;
    if (!token_range(p, b, t0, len, lane == 0 && jb == 0) || len == 0) continue;
    const int blk = t0 / p.bt + jb;
    const long long first = static_cast<long long>(blk) * p.bt;   // the block's first token
    const long long end = min(first + p.bt, static_cast<long long>(t0) + len);
    const long long lo = max(first, static_cast<long long>(t0));  // new rows: tokens lo .. end-1
    if (lo >= end) continue;
    const __nv_bfloat16* x = is_v ? p.v : p.k;
    uint8_t* codes = is_v ? p.v_codes : p.k_codes;
    const long long xrow = static_cast<long long>(p.n) * p.Hkv * D;  // elements of a token
    const long long xo = (static_cast<long long>(b) * p.L - t0) * xrow + (static_cast<long long>(s) * p.Hkv + hk) * D + col;
    const long long co = static_cast<long long>(b) * p.Tcap * xrow + (static_cast<long long>(s) * p.Hkv + hk) * D + col;
    const long long si = ((static_cast<long long>(b) * p.Hkv + hk) * p.nb + blk) * p.n + s;
    float* scale_ptr = (is_v ? p.v_scale : p.k_scale) + si;
    if (!in_bounds(si, 1, p.ext_scale, p.status)) continue;

    uint32_t am = 0;  // largest magnitude, as two bf16 halves
    for (long long t = lo + sub; t < end; t += RPP) {
      const long long o = xo + t * xrow;
      if (!in_bounds(o, 4, p.ext_rows, p.status)) continue;
      const uint2 r = __ldg(reinterpret_cast<const uint2*>(x + o));
      am = __vmaxu2(am, __vmaxu2(r.x & 0x7fff7fffu, r.y & 0x7fff7fffu));
    }
    const uint32_t abits = __reduce_max_sync(0xffffffffu, max(am & 0xffffu, am >> 16));
    const bool finite = abits < 0x7f80u;
    const float old = first < t0 ? *scale_ptr : 0.f;
    __syncwarp();  // every lane has read the old scale before lane 0 replaces it
    float now = finite ? fmaxf(scale_for<FMT>(abits), old) : __int_as_float(0x7fffffff);
    if (old != old) now = old;
    const bool poison = now != now;
    if (lane == 0) *scale_ptr = now;
    if (first < t0 && now > old) {
      for (long long t = first + sub; t < lo; t += RPP) {
        const long long o = co + t * xrow;
        if (!in_bounds(o, 4, p.ext_codes, p.status)) continue;
        uint32_t* c = reinterpret_cast<uint32_t*>(codes + o);
        *c = requantise4<FMT>(*c, old, now);
      }
    }
    const float inv = __fdiv_rn(1.f, now);
    for (long long t = lo + sub; t < end; t += RPP) {
      const long long o = xo + t * xrow, w = co + t * xrow;
      if (!in_bounds(o, 4, p.ext_rows, p.status) || !in_bounds(w, 4, p.ext_codes, p.status)) continue;
      const uint2 r = __ldg(reinterpret_cast<const uint2*>(x + o));
      *reinterpret_cast<uint32_t*>(codes + w) = poison ? 0u : quantise4<FMT>(r, inv);
    }
  }
}

// One thread a chunk of 8 codes: 8 bytes in, 16 bytes out.
template <int D, int FMT>
__global__ void __launch_bounds__(256) kv_read_q8_kernel(const KvQ8Params p) {
  constexpr int CPR = D / 8;
  const long long per_tensor = static_cast<long long>(p.B) * p.L * p.n * p.Hkv * CPR;
  const long long threads = static_cast<long long>(gridDim.x) * blockDim.x;
  for (long long u = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; u < 2 * per_tensor; u += threads) {
    const bool is_v = u >= per_tensor;
    const long long e = is_v ? u - per_tensor : u;  // chunk of the rows read
    long long i = e;
    const int ch = static_cast<int>(i % CPR);
    i /= CPR;
    const int hk = static_cast<int>(i % p.Hkv);
    i /= p.Hkv;
    const int s = static_cast<int>(i % p.n);
    i /= p.n;
    const int t = static_cast<int>(i % p.L);
    const int b = static_cast<int>(i / p.L);
    int t0, len;
    if (!token_range(p, b, t0, len, t == 0 && ch == 0) || t >= len) continue;
    const int tok = t0 + t;
    const long long co = (((static_cast<long long>(b) * p.Tcap + tok) * p.n + s) * p.Hkv + hk) * D + ch * 8;
    const long long si = ((static_cast<long long>(b) * p.Hkv + hk) * p.nb + tok / p.bt) * p.n + s;
    if (!in_bounds(co, 8, p.ext_codes, p.status) || !in_bounds(si, 1, p.ext_scale, p.status) ||
        !in_bounds(e * 8, 8, p.ext_rows, p.status))
      continue;
    const uint2 c = *reinterpret_cast<const uint2*>((is_v ? p.v_codes : p.k_codes) + co);
    const float sc = (is_v ? p.v_scale : p.k_scale)[si];
    uint32_t r[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t w = (j < 2 ? c.x : c.y) >> ((j & 1) * 16);
      r[j] = pack_bf16(code_value<FMT>(w & 0xffu) * sc, code_value<FMT>((w >> 8) & 0xffu) * sc);
    }
    *reinterpret_cast<uint4*>((is_v ? p.v_out : p.k_out) + e * 8) = make_uint4(r[0], r[1], r[2], r[3]);
  }
}

template <int D, int FMT>
cudaError_t launch_write_d(const KvQ8Params& p, int sms, cudaStream_t stream) {
  const long long units = 2LL * p.B * p.blocks * p.n * p.Hkv;
  long long grid = (units + kKvWarps - 1) / kKvWarps;
  const long long cap = static_cast<long long>(sms) * 8 * 16;
  if (grid > cap) grid = cap;
  kv_write_q8_kernel<D, FMT><<<static_cast<unsigned>(grid), kKvWarps * 32, 0, stream>>>(p);
  return cudaGetLastError();
}

template <int D, int FMT>
cudaError_t launch_read_d(const KvQ8Params& p, int sms, cudaStream_t stream) {
  const long long units = 2LL * p.B * p.L * p.n * p.Hkv * (D / 8);
  long long grid = (units + 255) / 256;
  const long long cap = static_cast<long long>(sms) * 8 * 16;
  if (grid > cap) grid = cap;
  kv_read_q8_kernel<D, FMT><<<static_cast<unsigned>(grid), 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_write_q8(const KvQ8Params& p, int sms, cudaStream_t stream) {
  const bool e4m3 = p.format == HD_Q8_E4M3;
  if (p.D == 64) return e4m3 ? launch_write_d<64, HD_Q8_E4M3>(p, sms, stream) : launch_write_d<64, HD_Q8_INT8>(p, sms, stream);
  if (p.D == 128) return e4m3 ? launch_write_d<128, HD_Q8_E4M3>(p, sms, stream) : launch_write_d<128, HD_Q8_INT8>(p, sms, stream);
  return cudaErrorInvalidValue;
}

cudaError_t launch_kv_read_q8(const KvQ8Params& p, int sms, cudaStream_t stream) {
  const bool e4m3 = p.format == HD_Q8_E4M3;
  if (p.D == 64) return e4m3 ? launch_read_d<64, HD_Q8_E4M3>(p, sms, stream) : launch_read_d<64, HD_Q8_INT8>(p, sms, stream);
  if (p.D == 128) return e4m3 ? launch_read_d<128, HD_Q8_E4M3>(p, sms, stream) : launch_read_d<128, HD_Q8_INT8>(p, sms, stream);
  return cudaErrorInvalidValue;
}

}  // namespace hd
