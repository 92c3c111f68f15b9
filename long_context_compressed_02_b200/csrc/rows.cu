// Row operators of a paged serving step: rotary positions, the norm of query
// and key rows with the rotation in the same pass, and the append of rows to a
// paged cache.
//
// For a row x at position p (gain g, frequencies w_j, magnitude c):
//   u = x * rsqrt(mean(x^2) + eps) * g                    (norm; else u = x)
//   (a, b) -> c (a cos p w_j - b sin p w_j, a sin p w_j + b cos p w_j)
// for the pairs (r0 + j, r0 + j + r/2) (half layout) or (r0 + 2j, r0 + 2j + 1)
// (interleaved), j < r/2; the other elements of u pass unchanged.
//
// All three move each row once and compute little, so memory bounds them: the
// large calls by HBM, the decode calls by latency.  A lane owns both elements of
// every pair that it rotates (see Unit), so a row needs no exchange but the sum
// of the norm.  The angles of a token are shared by all its rows: a CTA builds
// cos / sin once per token in shared memory while its first rows' loads are in
// flight.
#include <algorithm>
#include <cmath>
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include "common.cuh"
#include "tc.cuh"
#include "batch.cuh"

namespace csa {

static __device__ uint32_t g_err_rows;

uint32_t read_clear_err_rows() {
  uint32_t v = 0, z = 0;
  cudaMemcpyFromSymbol(&v, g_err_rows, sizeof(v));
  cudaMemcpyToSymbol(g_err_rows, &z, sizeof(z));
  return v;
}

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxTokens = kWarps;        // tokens per CTA: a warp looks up each

struct RowSetDesc {                       // rows x[i, h, :] of one tensor
  const void* x;
  void* y;
  const float* gain;                      // [D] or null
  int64_t x_tok, x_head, y_tok, y_head;   // strides in elements
  int H;
};

struct RowsParams {
  RowSetDesc set[2];                      // set 1 may have no rows (H = 0)
  const int32_t* cu_q;
  const int64_t* q_pos;
  int n_seq;
  int64_t n_tok;
  const double* inv_freq;                 // [r / 2]
  int D, r, r0, interleaved, norm;
  float sign, mscale, eps;                // sign -1: the inverse rotation
  int units, lpr;                         // units of a row, lanes per row (a power of two)
  int tpb, rows, rchunk;                  // tokens per CTA; rows per token; rows per CTA of each token
  // paged destination
  PageTable pt;
  uint8_t* nope;                          // e4m3 pages
  __nv_bfloat16* rope;
  float* scale;
};

enum Dest { DENSE = 0, PAGED = 1, PAGED_E4M3 = 2 };

// 8 consecutive elements
__device__ __forceinline__ void unpack8(const uint4 (&raw)[1], float* v) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(raw);
#pragma unroll
  for (int i = 0; i < 4; ++i) { const float2 f = __bfloat1622float2(h[i]); v[2 * i] = f.x; v[2 * i + 1] = f.y; }
}
__device__ __forceinline__ void unpack8(const uint4 (&raw)[2], float* v) {
  const float* f = reinterpret_cast<const float*>(raw);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = f[i];
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* v) {
  uint4 a;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&a);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
  *reinterpret_cast<uint4*>(p) = a;
}
__device__ __forceinline__ void store8(float* p, const float* v) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// A unit is two chunks of 8 elements.  The r / 16 rotated units come first:
// unit u holds chunks u and u + r / 16 of the rotated part, i.e. both halves of
// its pairs in the half layout (an interleaved pair lies within a chunk).  The
// remaining units hold chunks k and k + n / 2 of the n chunks outside the part.
// Consecutive lanes take consecutive chunks, so a warp's loads are whole lines.
struct Unit {
  int d[2];                               // first element of each chunk
  int j[2];                               // pair of the chunk's first element
  bool rot;
};
__device__ __forceinline__ Unit unit_of(const RowsParams& p, int u) {
  Unit w;
  const int ru = p.r >> 4;
  w.rot = u < ru;
  if (w.rot) {
    w.d[0] = p.r0 + 8 * u;
    w.d[1] = w.d[0] + (p.r >> 1);
    w.j[0] = p.interleaved ? 4 * u : 8 * u;
    w.j[1] = p.interleaved ? w.j[0] + (p.r >> 2) : w.j[0];
  } else {
    const int k = u - ru, n = (p.D - p.r) >> 3, before = p.r0 >> 3;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int c = k + i * (n >> 1);
      w.d[i] = 8 * (c < before ? c : c + (p.r >> 3));
      w.j[i] = 0;
    }
  }
  return w;
}

// UPL: units per lane; K: rows in flight per lane group.
template <typename Tin, typename Tout, int UPL, int K, int DEST>
__global__ void __launch_bounds__(kThreads)
rows_kernel(const __grid_constant__ RowsParams p) {
  constexpr int NV = sizeof(Tin) / 2;     // 16-byte vectors per chunk
  extern __shared__ float2 s_cs[];        // [tpb][r / 2]
  __shared__ int64_t s_pos[kMaxTokens];   // position, or -1: the token's rows are left alone
  __shared__ int s_seq[kMaxTokens];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t tok0 = (int64_t)blockIdx.x * p.tpb;
  const int row0 = blockIdx.y * p.rchunk;
  const int nr = min(p.rchunk, p.rows - row0);
  const int total = p.tpb * nr;
  const int gpw = 32 / p.lpr, gl = lane / p.lpr, ul = lane % p.lpr;

  Unit un[UPL];
  bool uv[UPL];
#pragma unroll
  for (int i = 0; i < UPL; ++i) {
    const int u = ul + i * p.lpr;
    uv[i] = u < p.units;
    un[i] = unit_of(p, uv[i] ? u : 0);
  }

  uint4 raw[K][UPL][2][NV];
  // Row `lr` of this CTA: token lr / nr, row row0 + lr % nr of its rows.
  auto load_rows = [&](int base) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int lr = base + k * kWarps * gpw;
      const int tl = lr / nr;
      if (lr >= total || tok0 + tl >= p.n_tok) continue;
      const int rr = row0 + lr % nr;
      const RowSetDesc& st = p.set[rr >= p.set[0].H];
      const int h = rr >= p.set[0].H ? rr - p.set[0].H : rr;
      const Tin* src = static_cast<const Tin*>(st.x) + (tok0 + tl) * st.x_tok + h * st.x_head;
#pragma unroll
      for (int i = 0; i < UPL; ++i)
        if (uv[i])
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int n = 0; n < NV; ++n) raw[k][i][c][n] = reinterpret_cast<const uint4*>(src + un[i].d[c])[n];
    }
  };
  const int first = warp * gpw + gl;
  load_rows(first);

  // positions: a warp looks up each token of the CTA
  if (warp < p.tpb) {
    const int64_t i = tok0 + warp;
    int b = -1;
    if (i < p.n_tok) b = find_seq_warp(p.cu_q, p.n_seq, i, lane);
    if (lane == 0) {
      s_seq[warp] = b;
      s_pos[warp] = b < 0 ? -1 : p.q_pos[b] + (i - p.cu_q[b]);
    }
  }
  __syncthreads();
  // Angles in double, reduced to [-pi, pi] there (positions reach 2^20 and
  // more), then cos and sin in float of the reduced angle.
  const int half = p.r >> 1;
  for (int e = tid; e < p.tpb * half; e += kThreads) {
    const int64_t pos = s_pos[e / half];
    if (pos < 0) continue;
    double a = (double)pos * p.inv_freq[e % half];
    a -= rint(a * 0.15915494309189533577) * 6.283185307179586477;
    float sn, cs;
    sincosf((float)a, &sn, &cs);
    s_cs[e] = make_float2(cs * p.mscale, sn * p.mscale * p.sign);
  }
  __syncthreads();

  for (int base = first; base - first < total; base += K * kWarps * gpw) {     // uniform over the CTA
    if (base != first) load_rows(base);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int lr = base + k * kWarps * gpw;
      const int tl = min(lr / nr, p.tpb - 1);
      const int rr = row0 + lr % nr;
      const int64_t pos = s_pos[tl];
      const bool on = lr < total && pos >= 0;
      const int si = rr >= p.set[0].H ? 1 : 0;
      const RowSetDesc& st = p.set[si];
      const int h = rr - (si ? p.set[0].H : 0);
      float v[UPL][16];
#pragma unroll
      for (int i = 0; i < UPL; ++i) {
        if (on && uv[i]) {
          unpack8(raw[k][i][0], v[i]);
          unpack8(raw[k][i][1], v[i] + 8);
        } else {
#pragma unroll
          for (int c = 0; c < 16; ++c) v[i][c] = 0.f;
        }
      }
      if (p.norm) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < UPL; ++i)
#pragma unroll
          for (int c = 0; c < 16; ++c) ss = fmaf(v[i][c], v[i][c], ss);
        for (int o = p.lpr >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float inv = rsqrtf(ss / (float)p.D + p.eps);
#pragma unroll
        for (int i = 0; i < UPL; ++i) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float4* g4 = reinterpret_cast<const float4*>(st.gain + un[i].d[c]);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const float4 g = st.gain ? __ldg(g4 + q) : make_float4(1.f, 1.f, 1.f, 1.f);
              float* w = v[i] + 8 * c + 4 * q;
              w[0] *= inv * g.x; w[1] *= inv * g.y; w[2] *= inv * g.z; w[3] *= inv * g.w;
            }
          }
        }
      }
#pragma unroll
      for (int i = 0; i < UPL; ++i) {
        if (!(on && un[i].rot)) continue;
        const float2* cs = s_cs + tl * half;
        if (p.interleaved) {
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 w = cs[un[i].j[c] + j];
              const float a = v[i][8 * c + 2 * j], b = v[i][8 * c + 2 * j + 1];
              v[i][8 * c + 2 * j] = a * w.x - b * w.y;
              v[i][8 * c + 2 * j + 1] = a * w.y + b * w.x;
            }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2 w = cs[un[i].j[0] + j];
            const float a = v[i][j], b = v[i][8 + j];
            v[i][j] = a * w.x - b * w.y;
            v[i][8 + j] = a * w.y + b * w.x;
          }
        }
      }
      if constexpr (DEST == DENSE) {
        if (on) {
          Tout* dst = static_cast<Tout*>(st.y) + (tok0 + tl) * st.y_tok + h * st.y_head;
#pragma unroll
          for (int i = 0; i < UPL; ++i)
            if (uv[i]) { store8(dst + un[i].d[0], v[i]); store8(dst + un[i].d[1], v[i] + 8); }
        }
      } else {
        int64_t row = -1;
        if (on) {
          row = page_row(p.pt, s_seq[tl], pos);
          if (row < 0 && ul == 0) atomicOr(&g_err_rows, DEV_ERR_BAD_INDEX);
        }
        if constexpr (DEST == PAGED) {
          if (row >= 0) {
            Tout* dst = static_cast<Tout*>(st.y) + row * p.D;
#pragma unroll
            for (int i = 0; i < UPL; ++i)
              if (uv[i]) { store8(dst + un[i].d[0], v[i]); store8(dst + un[i].d[1], v[i] + 8); }
          }
        } else {
          // s = max|.| / 448 over the D - r dims outside the rotated part
          float am = 0.f;
#pragma unroll
          for (int i = 0; i < UPL; ++i)
            if (uv[i] && !un[i].rot)
#pragma unroll
              for (int c = 0; c < 16; ++c) am = fmaxf(am, fabsf(v[i][c]));
          for (int o = p.lpr >> 1; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
          float s = am / 448.f;
          if (s == 0.f) s = 1.f;
          if (row >= 0) {
            if (ul == 0) p.scale[row] = s;
#pragma unroll
            for (int i = 0; i < UPL; ++i) {
              if (!uv[i]) continue;
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const float* w = v[i] + 8 * c;
                if (un[i].rot) {
                  store8(p.rope + row * p.r + (un[i].d[c] - p.r0), w);
                } else {
                  uint32_t q[2];
#pragma unroll
                  for (int n = 0; n < 2; ++n) {
                    const uint32_t a = __nv_cvt_float2_to_fp8x2(make_float2(w[4 * n] / s, w[4 * n + 1] / s), __NV_SATFINITE, __NV_E4M3);
                    const uint32_t b = __nv_cvt_float2_to_fp8x2(make_float2(w[4 * n + 2] / s, w[4 * n + 3] / s), __NV_SATFINITE, __NV_E4M3);
                    q[n] = a | (b << 16);
                  }
                  *reinterpret_cast<uint2*>(p.nope + row * (p.D - p.r) + un[i].d[c]) = make_uint2(q[0], q[1]);
                }
              }
            }
          }
        }
      }
    }
  }
}

template <typename Tin, typename Tout, int DEST>
csa_status_t launch_rows(RowsParams& p, const char* fn, cudaStream_t st) {
  p.rows = p.set[0].H + p.set[1].H;
  if (p.n_tok == 0 || p.rows == 0 || p.units == 0) return CSA_OK;
  p.lpr = 1;
  while (p.lpr < 32 && p.lpr < p.units) p.lpr *= 2;
  // about 32 rows a CTA: whole tokens if they have fewer rows, else an even part of one token's rows
  const int chunks = (p.rows + 32) / 33;
  p.rchunk = (p.rows + chunks - 1) / chunks;
  p.tpb = std::max(1, std::min(kMaxTokens, 32 / p.rows));
  if (p.r > 0) p.tpb = std::min(p.tpb, 8192 / p.r);      // angles within 32 KB (r is at most 2048)
  const int64_t gx = (p.n_tok + p.tpb - 1) / p.tpb;
  if (gx > 0x7fffffff || chunks > 65535) return fail(CSA_ERR_UNSUPPORTED, "%s: too many rows", fn);
  const dim3 grid((unsigned)gx, (unsigned)chunks);
  const size_t smem = (size_t)p.tpb * (p.r / 2) * sizeof(float2);
  const int upl = (p.units + p.lpr - 1) / p.lpr;
  cudaError_t e;
  if (upl == 1) e = launch_pdl(rows_kernel<Tin, Tout, 1, 4, DEST>, grid, dim3(kThreads), smem, st, p);
  else if (upl == 2) e = launch_pdl(rows_kernel<Tin, Tout, 2, 2, DEST>, grid, dim3(kThreads), smem, st, p);
  else e = launch_pdl(rows_kernel<Tin, Tout, 4, 1, DEST>, grid, dim3(kThreads), smem, st, p);
  if (e != cudaSuccess) return fail(CSA_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
  return check_launch(fn);
}

csa_status_t check_batch(const char* fn, const int32_t* cu_q, const int64_t* q_pos, int n_seq, int64_t n_tok) {
  CSA_REQUIRE(n_seq >= 0 && n_tok >= 0, "%s: n_seq and n_tok must not be negative", fn);
  CSA_REQUIRE(n_tok == 0 || n_seq == 0 || (cu_q && q_pos), "%s: cu_q and q_pos required", fn);
  CSA_REQUIRE(reinterpret_cast<uintptr_t>(cu_q) % 4 == 0 && reinterpret_cast<uintptr_t>(q_pos) % 8 == 0,
              "%s: cu_q / q_pos must be aligned to their elements", fn);
  return CSA_OK;
}

csa_status_t check_rows(const char* fn, int D, int r, int r0, const double* inv_freq, csa_dtype_t in, csa_dtype_t out) {
  CSA_REQUIRE(D % 16 == 0 && D >= 16 && D <= 2048, "%s: D must be a multiple of 16 in [16, 2048]", fn);
  CSA_REQUIRE(r >= 0 && r % 16 == 0 && r <= D, "%s: rope_dim must be a multiple of 16, at most D", fn);
  CSA_REQUIRE(r0 >= 0 && r0 % 8 == 0 && r0 + r <= D, "%s: rope_start must be a multiple of 8 with rope_start + rope_dim <= D", fn);
  CSA_REQUIRE(r == 0 || (inv_freq && reinterpret_cast<uintptr_t>(inv_freq) % 8 == 0), "%s: inv_freq required", fn);
  CSA_REQUIRE((in == CSA_F32 || in == CSA_BF16) && (out == CSA_F32 || out == CSA_BF16), "%s: dtypes must be F32 or BF16", fn);
  return CSA_OK;
}

// x rows readable and y rows writable by 16-byte vectors
csa_status_t check_set(const char* fn, const char* name, const RowSetDesc& s, csa_dtype_t in, csa_dtype_t out) {
  const int64_t ei = in == CSA_F32 ? 4 : 8, eo = out == CSA_F32 ? 4 : 8;      // elements of 16 bytes
  CSA_REQUIRE(s.x && s.y && aligned16(s.x) && aligned16(s.y), "%s: %s and its output must be non-null and 16-byte aligned", fn, name);
  CSA_REQUIRE(s.x_tok % ei == 0 && s.x_head % ei == 0 && s.y_tok % eo == 0 && s.y_head % eo == 0,
              "%s: strides of %s and its output must be multiples of 16 bytes", fn, name);
  CSA_REQUIRE(!s.gain || aligned16(s.gain), "%s: gain of %s must be 16-byte aligned", fn, name);
  return CSA_OK;
}

template <int DEST>
csa_status_t dispatch_rows(RowsParams& p, const char* fn, csa_dtype_t in, csa_dtype_t out, cudaStream_t st) {
  if (in == CSA_BF16)
    return out == CSA_BF16 ? launch_rows<__nv_bfloat16, __nv_bfloat16, DEST>(p, fn, st)
                           : launch_rows<__nv_bfloat16, float, DEST>(p, fn, st);
  return out == CSA_BF16 ? launch_rows<float, __nv_bfloat16, DEST>(p, fn, st) : launch_rows<float, float, DEST>(p, fn, st);
}

}  // namespace
}  // namespace csa

using namespace csa;

extern "C" csa_status_t csa_rope_freqs(int rope_dim, double base, double factor, double original_len, double beta_fast,
                                       double beta_slow, double* inv_freq, float* mscale) {
  clear_error();
  CSA_REQUIRE(rope_dim >= 2 && rope_dim % 2 == 0, "csa_rope_freqs: rope_dim must be even and positive");
  CSA_REQUIRE(base > 1.0 && std::isfinite(base), "csa_rope_freqs: base must be above 1");
  CSA_REQUIRE(factor >= 1.0 && std::isfinite(factor), "csa_rope_freqs: factor must be at least 1");
  CSA_REQUIRE(original_len >= 0.0 && std::isfinite(original_len), "csa_rope_freqs: original_len must not be negative");
  CSA_REQUIRE(original_len == 0.0 || beta_fast > beta_slow, "csa_rope_freqs: beta_fast must be above beta_slow");
  CSA_REQUIRE(inv_freq && mscale, "csa_rope_freqs: null output");
  for (int j = 0; j < rope_dim / 2; ++j) {
    const double w = std::pow(base, -2.0 * j / rope_dim);
    double keep = 0.0;                    // linear: every frequency is divided
    if (original_len > 0.0) {
      const double turns = original_len * w / 6.283185307179586477;
      keep = std::min(1.0, std::max(0.0, (turns - beta_slow) / (beta_fast - beta_slow)));
    }
    inv_freq[j] = keep * w + (1.0 - keep) * w / factor;
  }
  *mscale = original_len > 0.0 ? (float)(0.1 * std::log(factor) + 1.0) : 1.f;
  return CSA_OK;
}

extern "C" csa_status_t csa_rope(const void* x, csa_dtype_t in_dtype, int64_t x_tok_stride, int64_t x_head_stride,
                                 int64_t n_tok, int H, int D, const int32_t* cu_q, const int64_t* q_pos, int n_seq,
                                 const double* inv_freq, int rope_dim, int rope_start, int interleaved, int inverse,
                                 float mscale, void* out, csa_dtype_t out_dtype, int64_t out_tok_stride,
                                 int64_t out_head_stride, cudaStream_t stream) {
  clear_error();
  csa_status_t s = check_batch("csa_rope", cu_q, q_pos, n_seq, n_tok);
  if (s != CSA_OK) return s;
  CSA_REQUIRE(H >= 0, "csa_rope: H must not be negative");
  s = check_rows("csa_rope", D, rope_dim, rope_start, inv_freq, in_dtype, out_dtype);
  if (s != CSA_OK) return s;
  if (n_tok == 0 || H == 0 || n_seq == 0) return CSA_OK;
  RowsParams p{};
  p.set[0] = RowSetDesc{x, out, nullptr, x_tok_stride, x_head_stride, out_tok_stride, out_head_stride, H};
  s = check_set("csa_rope", "x", p.set[0], in_dtype, out_dtype);
  if (s != CSA_OK) return s;
  const bool in_place = x == out;
  CSA_REQUIRE(!in_place || (in_dtype == out_dtype && x_tok_stride == out_tok_stride && x_head_stride == out_head_stride),
              "csa_rope: out may be x only with x's dtype and strides");
  p.cu_q = cu_q; p.q_pos = q_pos; p.n_seq = n_seq; p.n_tok = n_tok; p.inv_freq = inv_freq;
  p.D = D; p.r = rope_dim; p.r0 = rope_start; p.interleaved = interleaved != 0; p.sign = inverse ? -1.f : 1.f;
  p.mscale = mscale;
  p.units = in_place ? rope_dim / 16 : D / 16;       // in place, only the rotated part is touched
  return dispatch_rows<DENSE>(p, "csa_rope", in_dtype, out_dtype, stream);
}

extern "C" csa_status_t csa_qk_norm_rope(const void* q, int64_t q_tok_stride, int64_t q_head_stride, int H, const void* k,
                                         int64_t k_tok_stride, int64_t k_head_stride, int Hk, csa_dtype_t in_dtype,
                                         int64_t n_tok, int D, const int32_t* cu_q, const int64_t* q_pos, int n_seq,
                                         const float* q_gain, const float* k_gain, float eps, const double* inv_freq,
                                         int rope_dim, int rope_start, int interleaved, float mscale, void* q_out,
                                         int64_t q_out_tok_stride, int64_t q_out_head_stride, void* k_out,
                                         int64_t k_out_tok_stride, int64_t k_out_head_stride, csa_dtype_t out_dtype,
                                         cudaStream_t stream) {
  clear_error();
  csa_status_t s = check_batch("csa_qk_norm_rope", cu_q, q_pos, n_seq, n_tok);
  if (s != CSA_OK) return s;
  CSA_REQUIRE(H >= 0 && Hk >= 0, "csa_qk_norm_rope: H and Hk must not be negative");
  CSA_REQUIRE(eps >= 0.f, "csa_qk_norm_rope: eps must not be negative");
  s = check_rows("csa_qk_norm_rope", D, rope_dim, rope_start, inv_freq, in_dtype, out_dtype);
  if (s != CSA_OK) return s;
  if (n_tok == 0 || n_seq == 0 || H + Hk == 0) return CSA_OK;
  RowsParams p{};
  p.set[0] = RowSetDesc{q, q_out, q_gain, q_tok_stride, q_head_stride, q_out_tok_stride, q_out_head_stride, H};
  p.set[1] = RowSetDesc{k, k_out, k_gain, k_tok_stride, k_head_stride, k_out_tok_stride, k_out_head_stride, Hk};
  for (int i = 0; i < 2; ++i) {
    if (p.set[i].H == 0) continue;
    s = check_set("csa_qk_norm_rope", i ? "k" : "q", p.set[i], in_dtype, out_dtype);
    if (s != CSA_OK) return s;
    CSA_REQUIRE(p.set[i].x != p.set[i].y || (in_dtype == out_dtype && p.set[i].x_tok == p.set[i].y_tok && p.set[i].x_head == p.set[i].y_head),
                "csa_qk_norm_rope: an output may be its input only with the same dtype and strides");
  }
  p.cu_q = cu_q; p.q_pos = q_pos; p.n_seq = n_seq; p.n_tok = n_tok; p.inv_freq = inv_freq;
  p.D = D; p.r = rope_dim; p.r0 = rope_start; p.interleaved = interleaved != 0; p.sign = 1.f; p.mscale = mscale;
  p.norm = 1; p.eps = eps; p.units = D / 16;
  return dispatch_rows<DENSE>(p, "csa_qk_norm_rope", in_dtype, out_dtype, stream);
}

extern "C" csa_status_t csa_paged_append(const void* rows, csa_dtype_t in_dtype, int64_t row_stride, int64_t n_tok, int D,
                                         const int32_t* cu_q, const int64_t* q_pos, int n_seq, const int32_t* block_table,
                                         int max_pages, int page_size, int64_t n_pages, int norm, const float* gain,
                                         float eps, const double* inv_freq, int rope_dim, int interleaved, float mscale,
                                         void* pages, csa_dtype_t page_dtype, void* pages_rope, float* pages_scale,
                                         cudaStream_t stream) {
  clear_error();
  csa_status_t s = check_batch("csa_paged_append", cu_q, q_pos, n_seq, n_tok);
  if (s != CSA_OK) return s;
  CSA_REQUIRE(page_dtype == CSA_F32 || page_dtype == CSA_BF16 || page_dtype == CSA_E4M3, "csa_paged_append: bad page_dtype");
  const bool e4m3 = page_dtype == CSA_E4M3;
  const csa_dtype_t out = e4m3 ? CSA_BF16 : page_dtype;
  s = check_rows("csa_paged_append", D, rope_dim, D - rope_dim, inv_freq, in_dtype, out);
  if (s != CSA_OK) return s;
  CSA_REQUIRE(page_size >= 1 && page_size <= 65536 && (page_size & (page_size - 1)) == 0,
              "csa_paged_append: page_size must be a power of two, at most 65536");
  CSA_REQUIRE(max_pages >= 1 && n_pages >= 1, "csa_paged_append: max_pages and n_pages must be positive");
  CSA_REQUIRE(eps >= 0.f, "csa_paged_append: eps must not be negative");
  CSA_REQUIRE(!e4m3 || (rope_dim == 64 && D > 64), "csa_paged_append: e4m3 pages need rope_dim 64 and D above 64");
  if (n_tok == 0 || n_seq == 0) return CSA_OK;
  CSA_REQUIRE(block_table && reinterpret_cast<uintptr_t>(block_table) % 4 == 0, "csa_paged_append: block_table required");
  CSA_REQUIRE(!e4m3 || (pages_rope && pages_scale && aligned16(pages_rope) && aligned16(pages_scale)),
              "csa_paged_append: e4m3 pages need pages_rope and pages_scale, 16-byte aligned");
  RowsParams p{};
  p.set[0] = RowSetDesc{rows, pages, gain, row_stride, 0, 0, 0, 1};
  s = check_set("csa_paged_append", "rows", p.set[0], in_dtype, out);
  if (s != CSA_OK) return s;
  p.cu_q = cu_q; p.q_pos = q_pos; p.n_seq = n_seq; p.n_tok = n_tok; p.inv_freq = inv_freq;
  p.D = D; p.r = rope_dim; p.r0 = D - rope_dim; p.interleaved = interleaved != 0; p.sign = 1.f; p.mscale = mscale;
  p.norm = norm != 0; p.eps = eps; p.units = D / 16;
  p.pt.table = block_table; p.pt.n_pages = n_pages; p.pt.max_pages = max_pages; p.pt.ps_log2 = __builtin_ctz((unsigned)page_size);
  p.nope = static_cast<uint8_t*>(pages); p.rope = static_cast<__nv_bfloat16*>(pages_rope); p.scale = pages_scale;
  if (e4m3)
    return in_dtype == CSA_BF16 ? launch_rows<__nv_bfloat16, __nv_bfloat16, PAGED_E4M3>(p, "csa_paged_append", stream)
                                : launch_rows<float, __nv_bfloat16, PAGED_E4M3>(p, "csa_paged_append", stream);
  return dispatch_rows<PAGED>(p, "csa_paged_append", in_dtype, out, stream);
}
