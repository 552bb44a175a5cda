// launch.h - internal host launchers (not part of the C ABI).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "hd_common.cuh"

namespace hd {

constexpr int kWinInf = 1 << 30;  // "no window": larger than any supported sequence

cudaError_t launch_attn_fwd_tc(const AttnParams& p, cudaStream_t stream);
cudaError_t launch_attn_bwd(const AttnParams& p, cudaStream_t stream);
cudaError_t launch_attn_bwd_tc_main(const AttnParams& p, cudaStream_t stream);

struct DecodeParams {
  const __nv_bfloat16* q;   // [B, nq, Hq, D]
  const __nv_bfloat16* kc;  // [B, Tcap*n, Hkv, D]
  const __nv_bfloat16* vc;
  const int32_t* seqlen;    // [B]
  __nv_bfloat16* o;         // [B, nq, Hq, D]
  float* lse;               // [B, Hq, nq]
  float* part_o;            // [B, Hkv, MT*16, splits, D] fp32
  float* part_ml;           // [B, Hkv, MT*16, splits, 2] fp32 (max in log2 units, sum)
  int* status;
  int B, n, Tcap, Hq, Hkv, D, mode, win;  // win = n*W or kWinInf
  // Query streams s0 .. s0+nq-1 of the new token (all n, or only the final one).
  int nq, s0;
  // Keys are indexed in a "key space": key index c is cache position
  // kres + c*kstride, and a sequence of T1 tokens holds T1*kpt keys. The whole
  // cache: (1, 0, n). The final stream alone (final-stream-only INTRA): (n, n-1, 1).
  int kstride, kres, kpt;
  int rows, mt, splits, chunk;             // rows = nq*(Hq/Hkv); chunk keys per split
  float scale_log2;
  // allocated elements, for the checked build's bounds checks
  long long ext_q;      // q, o: B * nq * Hq * D
  long long ext_lse;    // lse: B * Hq * nq
  long long ext_cache;  // each cache: B * Tcap * n * Hkv * D
  long long ext_part;   // partial rows: B * Hkv * mt * 16 * splits
};

// Number of splits / chunk length the decode launcher uses for `rows` query
// rows per (sequence, KV head) against up to `keys` keys on a GPU of `sms`
// streaming multiprocessors.
void decode_split_plan(int B, int rows, long long keys, int Hkv, int sms, int* mt, int* splits,
                       int* chunk);
cudaError_t launch_decode(const DecodeParams& p, cudaStream_t stream);

// Division of numbers below 2^31 by a divisor known at launch: with
// l = ceil(log2 d) and m = ceil(2^(31+l) / d), m is below 2^32 for d no power of
// two, and x / d = floor(x m / 2^(31+l)) as x (m d - 2^(31+l)) < 2^31 d <= 2^(31+l).
struct FastDiv {
  uint32_t mul, shift;  // mul = 0: a power of two
  static FastDiv by(uint32_t d) {
    FastDiv f = {0, 0};
    while ((1ull << f.shift) < d) ++f.shift;
    if ((1ull << f.shift) == d) return f;
    f.mul = static_cast<uint32_t>(((1ull << (31 + f.shift)) + d - 1) / d);
    f.shift -= 1;
    return f;
  }
  __host__ __device__ uint32_t div(uint32_t x) const {
    if (mul == 0) return x >> shift;
    return static_cast<uint32_t>((static_cast<unsigned long long>(x) * mul) >> 32) >> shift;
  }
};

// The 8-bit KV cache: rows written to or read from tokens t0 .. t0+len-1 of each
// sequence, t0 = token_offset[b] (or 0), len = lengths[b] (or L).
constexpr int kQ8MinExp = -60;  // the smallest scale is 2^-60
struct KvQ8Params {
  const __nv_bfloat16* k;  // write: [B, L*n, Hkv, D]
  const __nv_bfloat16* v;
  __nv_bfloat16* k_out;    // read: [B, L*n, Hkv, D]
  __nv_bfloat16* v_out;
  uint8_t* k_codes;        // [B, Tcap*n, Hkv, D]
  uint8_t* v_codes;
  float* k_scale;          // [B, Hkv, nb, n]
  float* v_scale;
  const int32_t* token_offset;  // [B] or null
  const int32_t* lengths;       // [B] or null
  int* status;
  int B, L, n, Tcap, Hkv, D, format, bt, nb;  // nb = blocks of bt tokens in Tcap
  int blocks;              // blocks that L tokens can touch
  int wpu;                 // warps of a (block, stream, head) of a write (set by the launcher)
  FastDiv div_hkv, div_n, div_bt;
  // allocated elements, for the checked build's bounds checks
  long long ext_rows, ext_codes, ext_scale;
};
cudaError_t launch_kv_write_q8(const KvQ8Params& p, cudaStream_t stream);
cudaError_t launch_kv_read_q8(const KvQ8Params& p, cudaStream_t stream);

// Decode attention over the 8-bit cache. The nq query streams s0 .. s0+nq-1 of
// the new token are `groups` problems a KV head of spg streams each: under INTRA
// one stream, whose keys are its tokens (kpt = 1); otherwise all of them, over
// the positions (kpt = n).
struct DecodeQ8Params {
  const __nv_bfloat16* q;   // [B, nq, Hq, D]
  const uint8_t* kc;        // [B, Tcap*n, Hkv, D]
  const uint8_t* vc;
  const float* ks;          // [B, Hkv, nb, n]
  const float* vs;
  const int32_t* seqlen;    // [B]
  __nv_bfloat16* o;         // [B, nq, Hq, D]
  float* lse;               // [B, Hq, nq]
  float* part_o;            // [mt, Hkv, slots, tile_rows, D] fp32
  float* part_ml;           // [mt, Hkv, slots, tile_rows, 2] fp32 (reference in log2 units, sum)
  int* status;
  int B, n, Tcap, Hq, Hkv, D, g, nq, s0, groups, spg, kpt;  // g = Hq / Hkv
  int win;                  // keys of the window (kWinInf: none)
  int rows, tile_rows, mt;  // rows = spg*g, in mt tiles of tile_rows
  // The line of rounds (of kQ8Round keys) of all problems of a KV head and row
  // tile: ctas pieces of it, of `least` rounds and more; whole: a problem a CTA instead
  int ctas, least, whole;
  int slots;                // parts of a line: B * groups + ctas
  int format, bt, nb;
  int step_stream, step_blk, step_off;  // how far a round moves a key's (stream, block, token in it)
  float scale_log2;
  FastDiv div_g, div_mt, div_groups, div_hkv, div_rows, div_n, div_bt;
  long long ext_q, ext_lse, ext_scale, ext_part;
};
constexpr int kQ8Round = 128;  // keys that a CTA's warps take at once
int decode_q8_tile_rows(int rows);
void decode_q8_plan(long long problems, long long most_keys, int D, int tile_rows, long long lines, int sms, int* ctas,
                    int* least, int* whole);
cudaError_t launch_decode_q8(const DecodeQ8Params& p, cudaStream_t stream);

struct RopeParams {
  __nv_bfloat16* q;             // [B, Sq, Hq, D] or null
  __nv_bfloat16* k;             // [B, S, Hkv, D] or null
  const int32_t* token_offset;  // [B] tokens before the call, or null (all 0)
  int* status;
  int B, S, Sq, n, Hq, Hkv, D, final_only;
  double log2_base;
};
cudaError_t launch_rope(const RopeParams& p, int sms, cudaStream_t stream);

struct LmHeadParams {
  const int32_t* labels;  // [R]
  float* loss;            // [R]
  float* lse;             // [R] or null
  float* part;            // [2][nvt][R]: per vocabulary tile max (log2 units), sum of exp2
  float* pick;            // [R] logit of the label
  int* status;
  long long R;            // rows (tokens) = B*L
  int V, d;
  int nrb, nvt;           // row pairs, vocabulary tiles (set by the launcher)
  long long units;
  // gradient pass only
  const float* lse_in;    // [R] natural-log LSE of the forward
  __nv_bfloat16* g;       // [R, g_ld] softmax - onehot, bf16
  long long g_ld;         // columns of g: V rounded up to 256
};
size_t lm_head_workspace_bytes(long long R, int V);
size_t lm_head_grad_workspace_bytes(long long R, int V);
cudaError_t launch_lm_head_ce_bwd(LmHeadParams p, const void* x, const void* w, int n, float scale,
                                  void* dh, float* dw, int num_sms, cudaStream_t stream);
cudaError_t launch_lm_head_ce(LmHeadParams p, const void* x, const void* w, int n, int num_sms,
                              cudaStream_t stream);
cudaError_t launch_final_readout(const void* x, void* out, long long rows, int n,
                                 long long row_bytes, int sms, int* status, cudaStream_t stream);

cudaError_t launch_wait_timeout(long long limit_cycles, int* status, cudaStream_t stream);

cudaError_t launch_expand(const int32_t* ids, const void* tables, void* out, int B, int L, int n,
                          int V, long long row_bytes, int sms, int* status, cudaStream_t stream);

}  // namespace hd
