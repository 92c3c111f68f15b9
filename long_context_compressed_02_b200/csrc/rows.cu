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
// of the norm.  Every warp is on its own: its task is a range of rows of one
// token, or the rows of a few tokens that have few; it issues the first rows'
// loads, then looks its tokens up and computes their angles once, shared by all
// the task's rows through its own part of shared memory.
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

constexpr int kMaxTokens = 8;             // tokens of a task
constexpr int kMaxWarps = 8;

struct RowSetDesc {                       // rows x[i, h, :] of one tensor
  const void* x;
  void* y;
  const float* gain;                      // [D] or null
  int64_t x_tok, x_head, y_tok, y_head;   // strides in elements
  int H;
  // tasks: tokens each; rows of each token; tasks that a group of tokens takes
  int tpt, rpt, chunks;
  int64_t tasks;
};

struct RowsParams {
  RowSetDesc set[2];                      // set 1 may have no rows (H = 0)
  const int32_t* cu_q;
  const int64_t* q_pos;
  int n_seq;
  int64_t n_tok;
  const double* inv_freq;                 // [r / 2]
  int D, r, r0, interleaved, norm;
  float sign, mscale, eps, inv_d;         // sign -1: the inverse rotation; inv_d = 1 / D
  int units, lpr;                         // units of a row, lanes per row (a power of two)
  int cs_per_warp;                        // shared-memory angles of a warp
  // paged destination
  PageTable pt;
  uint8_t* nope;                          // e4m3 pages
  __nv_bfloat16* rope;
  float* scale;
};

enum Dest { DENSE = 0, PAGED = 1, PAGED_E4M3 = 2 };

// Two float32 operations in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(reinterpret_cast<unsigned long long&>(r))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(reinterpret_cast<unsigned long long&>(r))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)),
        "l"(reinterpret_cast<unsigned long long&>(c)));
  return r;
}

// 8 consecutive elements as 4 pairs
__device__ __forceinline__ void unpack8(const uint4 (&raw)[1], float2* v) {
  const uint32_t w[4] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
__device__ __forceinline__ void unpack8(const uint4 (&raw)[2], float2* v) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    v[2 * i] = make_float2(__uint_as_float(raw[i].x), __uint_as_float(raw[i].y));
    v[2 * i + 1] = make_float2(__uint_as_float(raw[i].z), __uint_as_float(raw[i].w));
  }
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float2* v) {
  uint4 a;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&a);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __float22bfloat162_rn(v[i]);
  *reinterpret_cast<uint4*>(p) = a;
}
__device__ __forceinline__ void store8(float* p, const float2* v) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
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

// Sequence of token i by one thread, -1 if it has none.
__device__ __forceinline__ int find_seq(const int32_t* cu_q, int n_seq, int64_t i) {
  if (i < cu_q[0] || i >= cu_q[n_seq]) return -1;
  int lo = 0, hi = n_seq;                 // the last b with cu_q[b] <= i
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu_q[mid] <= i) lo = mid; else hi = mid;
  }
  return lo;
}

// UPL: units per lane; K: row groups (32 / lpr rows) in flight per warp.
// Two groups and 24 warps an SM (80 registers) were the best of the measured
// splits: 4,850 tokens of 64 + 1 rows of 512 bf16 take 122 us (5.4 TB/s, 0.82 of
// the copy rate; the bf16 instances spill up to 9 registers) against 168 us with 32
// warps (64 registers, more spills) and 162 us with four groups and 16 warps;
// 11,700 tokens of 64 rows of 128, turned whole, 76 us (5.35 TB/s).  The issue
// slots, not DRAM, were full before the float32 pairs (mul2, fma2) and the shared
// look-ups: 390 instructions a row, 142 us.  Appended prompt rows share no look-up:
// 26,900 of 512 take 18 us into bf16 pages (12 us without the rotation) and 21 us into
// e4m3 pages, with 59 and 64 % of the issue slots taken while they run.
template <typename Tin, typename Tout, int UPL, int K, int DEST>
__global__ void __launch_bounds__(32 * kMaxWarps, UPL == 4 ? 1 : sizeof(Tin) * UPL > 2 ? 2 : 3)
rows_kernel(const __grid_constant__ RowsParams p) {
  constexpr int NV = sizeof(Tin) / 2;     // 16-byte vectors per chunk
  extern __shared__ float2 s_angles[];    // [warps][cs_per_warp]
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t task = (int64_t)blockIdx.x * (blockDim.x >> 5) + warp;
  const int si = task >= p.set[0].tasks;
  const RowSetDesc& st = p.set[si];
  if (si) task -= p.set[0].tasks;
  if (task >= st.tasks) return;           // warps do not wait for one another
  const int64_t tok0 = task / st.chunks * st.tpt;
  const int h0 = (int)(task % st.chunks) * st.rpt;
  const int nr = min(st.rpt, st.H - h0);
  const int nt = (int)min((int64_t)st.tpt, p.n_tok - tok0);
  const int total = nt * nr;
  const int gpw = 32 / p.lpr, gl = lane / p.lpr, ul = lane % p.lpr;
  const Tin* x0 = static_cast<const Tin*>(st.x) + tok0 * st.x_tok + h0 * st.x_head;

  Unit un[UPL];
  bool uv[UPL];
#pragma unroll
  for (int i = 0; i < UPL; ++i) {
    const int u = ul + i * p.lpr;
    uv[i] = u < p.units;
    un[i] = unit_of(p, uv[i] ? u : 0);
  }

  // Row lr of the task: token tok0 + lr / nr, head h0 + lr % nr.  K row groups
  // are in flight: a group's registers are refilled as soon as it is unpacked.
  // lr / nr by a product: the task's lr and the K groups ahead stay below 1024, and
  // nr at most 256 where a task has several tokens, so rcp is less than 256 2^-20 / nr
  // too large and lr times that does not reach the next 1 / nr
  const uint32_t rcp = nt == 1 ? 0 : ((1u << 20) - 1 + nr) / nr;
  auto token_of = [&](int lr) { return (int)(((uint32_t)lr * rcp) >> 20); };
  uint4 raw[K][UPL][2][NV];
  auto load_row = [&](int k, int lr) {
    if (lr >= total) return;
    const int tl = token_of(lr);
    const Tin* src = x0 + tl * st.x_tok + (lr - tl * nr) * st.x_head;
#pragma unroll
    for (int i = 0; i < UPL; ++i)
      if (uv[i])
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int n = 0; n < NV; ++n) raw[k][i][c][n] = reinterpret_cast<const uint4*>(src + un[i].d[c])[n];
  };
#pragma unroll
  for (int k = 0; k < K; ++k) load_row(k, gl + k * gpw);

  // the gains of a lane's only unit stay in registers
  auto load_gain = [&](int d) {
    return __ldg(reinterpret_cast<const float4*>(st.gain + d));
  };
  float4 gain[4];
  if (UPL == 1 && st.gain)
#pragma unroll
    for (int c = 0; c < 4; ++c) gain[c] = load_gain(un[0].d[c >> 1] + 4 * (c & 1));

  // lane l < nt: sequence and position of token tok0 + l; position -1: its rows are left alone
  int seq = -1;
  int64_t pos = -1, slot = -1;            // slot: its row of the page store
  if (lane < nt) {
    seq = find_seq(p.cu_q, p.n_seq, tok0 + lane);
    if (seq >= 0) pos = p.q_pos[seq] + (tok0 + lane - p.cu_q[seq]);
    if (DEST != DENSE && pos >= 0) {
      slot = page_row(p.pt, seq, pos);
      if (slot < 0) atomicOr(&g_err_rows, DEV_ERR_BAD_INDEX);
    }
  }
  // Angles in double (positions reach 2^20 and more), as the part of a turn in
  // [-1/2, 1/2], then cos and sin in float of that part times 2 pi.
  float2* s_cs = s_angles + warp * p.cs_per_warp;
  const int half = p.r >> 1;
  for (int e0 = 0; e0 < nt * half; e0 += 32) {
    const int e = e0 + lane;
    const int tl = e / half;
    const int64_t ps = __shfl_sync(0xffffffffu, pos, tl & 31);
    if (e < nt * half) {
      const double turns = (double)ps * p.inv_freq[e - tl * half] * 0.15915494309189533577;
      float sn, cs;
      sincospif((float)(2.0 * (turns - rint(turns))), &sn, &cs);
      s_cs[e] = make_float2(cs * p.mscale, sn * p.mscale * p.sign);
    }
  }
  __syncwarp();

  for (int base = gl; base - gl < total; base += K * gpw) {     // uniform over the warp
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (base - gl + k * gpw >= total) break;                  // uniform too
      const int lr = base + k * gpw;
      const int tl = token_of(lr) & 31;
      const int64_t ps = __shfl_sync(0xffffffffu, pos, tl);
      const bool on = lr < total && ps >= 0;
      float2 v[UPL][8];
#pragma unroll
      for (int i = 0; i < UPL; ++i) {
        if (uv[i]) {
          unpack8(raw[k][i][0], v[i]);
          unpack8(raw[k][i][1], v[i] + 4);
        } else {
#pragma unroll
          for (int c = 0; c < 8; ++c) v[i][c] = make_float2(0.f, 0.f);
        }
      }
      load_row(k, lr + K * gpw);
      if (p.norm) {
        float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < UPL; ++i)
#pragma unroll
          for (int c = 0; c < 8; ++c) s2 = fma2(v[i][c], v[i][c], s2);
        float ss = s2.x + s2.y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          const float t = __shfl_xor_sync(0xffffffffu, ss, o);
          if (o < p.lpr) ss += t;
        }
        const float inv = rsqrtf(fmaf(ss, p.inv_d, p.eps));
#pragma unroll
        for (int i = 0; i < UPL; ++i)
#pragma unroll
          for (int c = 0; c < 8; ++c) v[i][c] = mul2(v[i][c], make_float2(inv, inv));
        if (st.gain) {
#pragma unroll
          for (int i = 0; i < UPL; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const float4 g = UPL == 1 ? gain[c] : load_gain(un[i].d[c >> 1] + 4 * (c & 1));
              v[i][2 * c] = mul2(v[i][2 * c], make_float2(g.x, g.y));
              v[i][2 * c + 1] = mul2(v[i][2 * c + 1], make_float2(g.z, g.w));
            }
        }
      }
#pragma unroll
      for (int i = 0; i < UPL; ++i) {
        if (!(on && un[i].rot)) continue;
        // (cos, sin) of two pairs at a time
        const float4* cs = reinterpret_cast<const float4*>(s_cs + tl * half);
        if (p.interleaved) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float4 w = cs[(un[i].j[c >> 1] >> 1) + (c & 1)];
            float2& e = v[i][2 * c];
            float2& f = v[i][2 * c + 1];
            e = make_float2(e.x * w.x - e.y * w.y, e.x * w.y + e.y * w.x);
            f = make_float2(f.x * w.z - f.y * w.w, f.x * w.w + f.y * w.z);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float4 w = cs[(un[i].j[0] >> 1) + j];
            const float2 c2 = make_float2(w.x, w.z), s2 = make_float2(w.y, w.w);
            const float2 a = v[i][j], b = v[i][4 + j];
            v[i][j] = fma2(a, c2, mul2(b, make_float2(-s2.x, -s2.y)));
            v[i][4 + j] = fma2(b, c2, mul2(a, s2));
          }
        }
      }
      if constexpr (DEST == DENSE) {
        if (on) {
          Tout* dst = static_cast<Tout*>(st.y) + (tok0 + tl) * st.y_tok + (h0 + lr - tl * nr) * st.y_head;
#pragma unroll
          for (int i = 0; i < UPL; ++i)
            if (uv[i]) { store8(dst + un[i].d[0], v[i]); store8(dst + un[i].d[1], v[i] + 4); }
        }
      } else {
        const int64_t at = __shfl_sync(0xffffffffu, slot, tl);
        const int64_t row = on ? at : -1;
        if constexpr (DEST == PAGED) {
          if (row >= 0) {
            Tout* dst = static_cast<Tout*>(st.y) + row * p.D;
#pragma unroll
            for (int i = 0; i < UPL; ++i)
              if (uv[i]) { store8(dst + un[i].d[0], v[i]); store8(dst + un[i].d[1], v[i] + 4); }
          }
        } else {
          // s = max|.| / 448 over the D - r dims outside the rotated part
          float am = 0.f;
#pragma unroll
          for (int i = 0; i < UPL; ++i)
            if (uv[i] && !un[i].rot)
#pragma unroll
              for (int c = 0; c < 8; ++c) am = fmaxf(am, fmaxf(fabsf(v[i][c].x), fabsf(v[i][c].y)));
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) {
            const float t = __shfl_xor_sync(0xffffffffu, am, o);
            if (o < p.lpr) am = fmaxf(am, t);
          }
          float s = am / 448.f;
          if (s == 0.f) s = 1.f;
          // one division a row, not one an element; rows so small that the
          // inverse would overflow are scaled up first
          float rs = 1.f / s;
          if (s < 1e-37f) {
            rs = 1.f / (s * 0x1p60f);
#pragma unroll
            for (int i = 0; i < UPL; ++i)
              if (!un[i].rot)
#pragma unroll
                for (int c = 0; c < 8; ++c) v[i][c] = mul2(v[i][c], make_float2(0x1p60f, 0x1p60f));
          }
          if (row >= 0) {
            if (ul == 0) p.scale[row] = s;
#pragma unroll
            for (int i = 0; i < UPL; ++i) {
              if (!uv[i]) continue;
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                if (un[i].rot) {
                  store8(p.rope + row * p.r + (un[i].d[c] - p.r0), v[i] + 4 * c);
                } else {
                  uint32_t q[2];
#pragma unroll
                  for (int n = 0; n < 2; ++n) {
                    const float2 r2 = make_float2(rs, rs);
                    const uint32_t lo = __nv_cvt_float2_to_fp8x2(mul2(v[i][4 * c + 2 * n], r2), __NV_SATFINITE, __NV_E4M3);
                    const uint32_t hi = __nv_cvt_float2_to_fp8x2(mul2(v[i][4 * c + 2 * n + 1], r2), __NV_SATFINITE, __NV_E4M3);
                    q[n] = lo | (hi << 16);
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
  if (p.n_tok == 0 || p.set[0].H + p.set[1].H == 0 || p.units == 0) return CSA_OK;
  p.lpr = 1;
  while (p.lpr < 32 && p.lpr < p.units) p.lpr *= 2;
  const int upl = (p.units + p.lpr - 1) / p.lpr;
  const int per_pass = 32 / p.lpr * (upl == 1 ? 2 : 1);   // rows in flight of a warp
  const int warps_wanted = num_sms() * 16;
  p.inv_d = 1.f / (float)p.D;
  p.cs_per_warp = 0;
  int64_t tasks = 0;
  for (RowSetDesc& s : p.set) {
    s.tasks = 0;
    s.tpt = s.rpt = s.chunks = 1;
    if (s.H == 0) continue;
    // A task has up to eight passes of rows, which share their token's look-up and
    // angles; fewer where that leaves warps idle, so that a small batch is over
    // sooner.
    int want = 8 * per_pass;
    while (want > per_pass && p.n_tok * s.H / want < warps_wanted) want /= 2;
    if (want < per_pass) want = per_pass;
    if (s.H >= want) {
      s.chunks = (s.H + want - 1) / want;
      s.rpt = (s.H + s.chunks - 1) / s.chunks;
      s.chunks = (s.H + s.rpt - 1) / s.rpt;
    } else {
      s.rpt = s.H;
      s.tpt = std::max(1, std::min(kMaxTokens, want / s.H));
      while (s.tpt > 1 && (s.tpt * p.r > 1024 || p.n_tok * s.H / (s.tpt * s.H) < warps_wanted / 2)) --s.tpt;
    }
    s.tasks = (p.n_tok + s.tpt - 1) / s.tpt * s.chunks;
    tasks += s.tasks;
    p.cs_per_warp = std::max(p.cs_per_warp, s.tpt * (p.r / 2));
  }
  int warps = kMaxWarps;
  while (warps > 1 && warps * p.cs_per_warp * sizeof(float2) > 32768) warps /= 2;
  // a small batch spreads over all SMs
  while (warps > 1 && tasks / warps < num_sms()) warps /= 2;
  const int64_t gx = (tasks + warps - 1) / warps;
  if (gx > 0x7fffffff) return fail(CSA_ERR_UNSUPPORTED, "%s: too many rows", fn);
  const dim3 grid((unsigned)gx), block(32 * warps);
  const size_t smem = (size_t)warps * p.cs_per_warp * sizeof(float2);
  cudaError_t e;
  if (upl == 1) e = launch_pdl(rows_kernel<Tin, Tout, 1, 2, DEST>, grid, block, smem, st, p);
  else if (upl == 2) e = launch_pdl(rows_kernel<Tin, Tout, 2, 1, DEST>, grid, block, smem, st, p);
  else e = launch_pdl(rows_kernel<Tin, Tout, 4, 1, DEST>, grid, block, smem, st, p);
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
