// selective_cache_kernels.cuh -- the selective scan of selective_kernels.cuh as a server runs it:
// over a packed batch of prompts of different lengths, and for one token of each sequence, with
// the states in a cache and the step's softplus and the output gate in the same kernel.
// "Architektury Mamba-2, State Space Models i liniowa atencja" (tech.tersel.eu), section "Od S4
// do Mamba-1: Wprowadzenie mechanizmu selektywnego"; "State Space Models (SSM)" (ultralytics.com
// glossary), sections "Come funzionano gli SSM" (the recurrent form) and "Da S4 a Mamba" (the
// SiLU gate).  Per sequence and channel d of group g:
//
//   dt = softplus(raw_t[d] + bias[d])            (or raw + bias as given)
//   h[n] <- exp(dt A[d,n]) h[n] + dt x_t[d] B_t[g,n]
//   y_t[d] = (sum_n C_t[g,n] h[n] + D[d] x_t[d]) * silu(z_t[d])
//
// Every (token, channel, state) needs its own exponential: dstate ex2 per token and channel at
// 16 per clock and SM bound the prompts' kernel; the token kernel streams the states.
#pragma once
#include "conv_cache_kernels.cuh"

namespace ssd {
namespace cache {

struct SelArgs {
  const void* x;
  const void* dt;
  const float* A;
  const void* B;
  const void* C;
  const float* D;
  const float* dt_bias;
  const void* z;
  void* y;
  float* state;
  const int* cu;
  const int* slots;
  const unsigned char* resume;
  float* ws_state;  // [units, dim, dstate]: the state after each chunk (long sequences only)
  float* ws_dt;     // [units, dim]: its sum of dt
  int64_t xs, dts, bs, cs, zs, ys;  // row strides in elements
  int64_t ntok, nslots;
  int nseq, dim, dstate, ngroups;
  int chunk;   // tokens per unit (0: a unit is a whole sequence)
  int nunits;  // units the workspace has room for: ntok / chunk + nseq
  bool io_bf16, dt_bf16, y_bf16, softplus;
};

// Decay rates in log2 units; a rate of -inf is held finite, so that an identity step (dt = 0)
// leaves the state and does not make a NaN of it.
__device__ __forceinline__ float rate2(float a) {
  const float r = a * kLog2e;
  return r < -1e38f ? -1e38f : r;
}

// softplus(v) = max(v, 0) + log(1 + e^-|v|): no exponential overflows, and small results keep
// their relative accuracy through log1p.
__device__ __forceinline__ float softplus_acc(float v) {
  return fmaxf(v, 0.f) + log1pf(expf(-fabsf(v)));
}

__device__ __forceinline__ float load_any(const void* p, int64_t i, bool bf16) {
  return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i])
              : static_cast<const float*>(p)[i];
}

// LPC lanes per channel, each holding 4 of its (up to 4 LPC) states; R channels per lane.
template <int LPC, int R>
struct SelShape {
  static constexpr int kCg = 32 / LPC;         // channel sets of a warp
  static constexpr int kCh = kCg * R;          // channels of a warp
  static constexpr int kNp = LPC * 4;          // states, padded
  static constexpr int kTok = LPC <= 4 ? 16 : 8;  // tokens staged together
  static constexpr int kDu = 2 * kCh + 4;      // floats per staged row of (dt, dt x) pairs
  static constexpr int kY = kCh + 8;           // and of y
  static constexpr int kEx = kTok * kCh / 32;  // x, dt, z elements per lane and stage
  static constexpr int kEb = kTok * kNp / 32;  // B, C elements per lane and stage
  static constexpr int kFloats = kTok * (kDu + 2 * kNp + kY);
  static_assert(kTok * kCh % 32 == 0 && 32 % kCh == 0, "whole rows per step of the warp");
};

// One warp scans one unit: a sequence (chunk == 0) or a chunk of one, for kCh channels of one
// group.  SUMMARY: only the state after the chunk, from zero (or, for a sequence's first chunk,
// from the sequence's initial state), and the chunk's sum of dt; those give the scan of a later
// chunk its entering state, h <- exp(A sum_dt) h + S chunk by chunk.
//
// Inputs come in stages of kTok tokens: the next stage's loads are issued into registers ahead
// of the current stage's steps, then converted (softplus, dt x, D x) once per element into
// shared memory, where the lanes of a channel all read them.  Neighbouring lanes load
// neighbouring channels element by element, so no alignment is asked of the rows.
template <int LPC, int R, bool SUMMARY>
__global__ void __launch_bounds__(32) selective_varlen_kernel(const SelArgs a) {
  using S = SelShape<LPC, R>;
  constexpr int TK = S::kTok, CH = S::kCh, NP = S::kNp;
  __shared__ __align__(16) float sm[S::kFloats];
  float* du = sm;
  float* bsm = du + TK * S::kDu;
  float* csm = bsm + TK * NP;
  float* ysm = csm + TK * NP;

  const int lane = threadIdx.x;
  const int dpg = a.dim / a.ngroups;
  const int cpg = (dpg + CH - 1) / CH;  // channel blocks per group
  const unsigned ncb = unsigned(cpg) * a.ngroups;
  const int unit = int(blockIdx.x / ncb), cb = int(blockIdx.x % ncb);
  const int g = cb / cpg;
  const int d0 = g * dpg + (cb % cpg) * CH;  // first channel
  const int nch = min(CH, (g + 1) * dpg - d0);
  const int N = a.dstate;

  if (!SUMMARY && blockIdx.x == 0) warp_check_seqs(a.cu, a.nseq, a.ntok);

  // the unit's sequence, and its chunk within the sequence
  int seq = unit, chunk = 0, nchunk = 1;
  if (a.chunk) {
    seq = -1;
    int base = 0;
    for (int i0 = 0; i0 < a.nseq && seq < 0; i0 += 32) {
      const int i = i0 + lane;
      int n = 0;
      if (i < a.nseq) {
        const int64_t len = int64_t(a.cu[i + 1]) - a.cu[i];
        n = len <= 0 ? 1 : int((min(len, a.ntok) + a.chunk - 1) / a.chunk);
      }
      int incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      const unsigned m = __ballot_sync(0xffffffffu, unit < base + incl && i < a.nseq);
      if (m) {
        const int l = __ffs(m) - 1;
        seq = i0 + l;
        nchunk = __shfl_sync(0xffffffffu, n, l);
        chunk = unit - (base + __shfl_sync(0xffffffffu, incl, l) - nchunk);
      }
      base = min(base + __shfl_sync(0xffffffffu, incl, 31), 1 << 30);
    }
    // bounds that do not increase can name more chunks than there is room for (latched above)
    if (seq < 0 || unit - chunk + nchunk > a.nunits) return;
  }
  if (SUMMARY && nchunk == 1) return;
  const int64_t s0 = a.cu[seq], s1 = a.cu[seq + 1];
  if (s0 < 0 || s1 < s0 || s1 > a.ntok) return;
  const int64_t slot = a.state || a.slots ? warp_slot(a.slots, seq, a.nslots) : 0;
  if (slot < 0) return;
  const bool last = chunk == nchunk - 1;
  const bool resume = a.state && a.resume && a.resume[seq];

  // this lane's channels, states and constants
  const int q = lane % LPC, cg = lane / LPC;
  float2 a01[R], a23[R], h01[R], h23[R];
  float sdt[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int c = cg * R + r;
    float av[4], hv[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int n = q * 4 + k;
      const bool on = c < nch && n < N;
      av[k] = on ? rate2(a.A[int64_t(d0 + c) * N + n]) : 0.f;
      hv[k] = on && resume && chunk == 0 && (SUMMARY || nchunk == 1)
                  ? a.state[(slot * a.dim + d0 + c) * N + n] : 0.f;
      if (on && !SUMMARY && nchunk > 1) {
        // a sequence cut into chunks: its initial state was copied by the summary launch (the
        // last chunk may already have moved the slot's), the others' follow from the summaries
        const int64_t u0 = unit - chunk;
        if (chunk == 0) {
          if (resume) hv[k] = a.ws_state[((u0 + nchunk - 1) * a.dim + d0 + c) * N + n];
        } else {
          float h = a.ws_state[(u0 * a.dim + d0 + c) * N + n];
          for (int j = 1; j < chunk; ++j)
            h = fmaf(ex2(av[k] * a.ws_dt[(u0 + j) * a.dim + d0 + c]), h,
                     a.ws_state[((u0 + j) * a.dim + d0 + c) * N + n]);
          hv[k] = h;
        }
      }
      if (on && SUMMARY && chunk == 0 && resume)
        a.ws_state[(int64_t(unit + nchunk - 1) * a.dim + d0 + c) * N + n] = hv[k];
    }
    a01[r] = make_float2(av[0], av[1]);
    a23[r] = make_float2(av[2], av[3]);
    h01[r] = make_float2(hv[0], hv[1]);
    h23[r] = make_float2(hv[2], hv[3]);
    sdt[r] = 0.f;
  }
  if (SUMMARY && last) return;

  const int64_t t0 = s0 + int64_t(chunk) * a.chunk;
  const int64_t t1 = a.chunk && t0 + a.chunk < s1 ? t0 + a.chunk : s1;

  // staging: element e = i * 32 + lane of a stage's [TK][CH] (or [TK][NP]) tile
  const int ec = lane % CH, et = lane / CH;  // channel and first token row of x, dt, z, y
  const bool eon = ec < nch;
  const float Dd = eon && a.D ? a.D[d0 + ec] : 0.f;
  const float bias = eon && a.dt_bias ? a.dt_bias[d0 + ec] : 0.f;
  constexpr int kRows = 32 / CH;  // token rows per step of the warp
  float rx[S::kEx], rd[S::kEx], rz[S::kEx], zc[S::kEx], rb[S::kEb], rc[S::kEb];
  auto load = [&](int64_t t) {
#pragma unroll
    for (int i = 0; i < S::kEx; ++i) {
      const int64_t tt = t + et + i * kRows;
      const bool on = eon && tt < t1;
      rx[i] = on ? load_any(a.x, tt * a.xs + d0 + ec, a.io_bf16) : 0.f;
      rd[i] = on ? load_any(a.dt, tt * a.dts + d0 + ec, a.dt_bf16) : 0.f;
      if (!SUMMARY) rz[i] = on && a.z ? load_any(a.z, tt * a.zs + d0 + ec, a.io_bf16) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < S::kEb; ++i) {
      const int e = i * 32 + lane, n = e % NP;
      const int64_t tt = t + e / NP;
      const bool on = n < N && tt < t1;
      rb[i] = on ? load_any(a.B, tt * a.bs + int64_t(g) * N + n, a.io_bf16) : 0.f;
      if (!SUMMARY) rc[i] = on ? load_any(a.C, tt * a.cs + int64_t(g) * N + n, a.io_bf16) : 0.f;
    }
  };
  auto stage = [&](int64_t t) {
#pragma unroll
    for (int i = 0; i < S::kEx; ++i) {
      const int row = et + i * kRows;
      float dt = rd[i] + bias;
      if (a.softplus) dt = softplus_acc(dt);
      const bool on = t + row < t1;  // rows past the end are identity steps
      *reinterpret_cast<float2*>(du + row * S::kDu + 2 * ec) =
          on ? make_float2(dt, dt * rx[i]) : make_float2(0.f, 0.f);
      if (!SUMMARY) {
        ysm[row * S::kY + ec] = Dd * rx[i];
        zc[i] = rz[i];
      }
    }
#pragma unroll
    for (int i = 0; i < S::kEb; ++i) {
      bsm[i * 32 + lane] = rb[i];
      if (!SUMMARY) csm[i * 32 + lane] = rc[i];
    }
  };

  if (t0 < t1) {
    load(t0);
    stage(t0);
  }
  __syncwarp();
  for (int64_t t = t0; t < t1; t += TK) {
    if (t + TK < t1) load(t + TK);
    const int steps = t1 - t < TK ? int((t1 - t + 3) / 4) : TK / 4;
    for (int k4 = 0; k4 < steps; ++k4) {
      float pv[R][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = k4 * 4 + i;
        const float4 bv = *reinterpret_cast<const float4*>(bsm + row * NP + q * 4);
        float4 cv;
        if (!SUMMARY) cv = *reinterpret_cast<const float4*>(csm + row * NP + q * 4);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float2 v =
              *reinterpret_cast<const float2*>(du + row * S::kDu + 2 * (cg * R + r));
          const float2 dd = make_float2(v.x, v.x), uu = make_float2(v.y, v.y);
          const float2 l01 = mul2(dd, a01[r]), l23 = mul2(dd, a23[r]);
          h01[r] = fma2(make_float2(ex2(l01.x), ex2(l01.y)), h01[r],
                        mul2(uu, make_float2(bv.x, bv.y)));
          h23[r] = fma2(make_float2(ex2(l23.x), ex2(l23.y)), h23[r],
                        mul2(uu, make_float2(bv.z, bv.w)));
          if (SUMMARY) {
            sdt[r] += v.x;
          } else {
            const float2 p = fma2(make_float2(cv.z, cv.w), h23[r],
                                  mul2(make_float2(cv.x, cv.y), h01[r]));
            pv[r][i] = p.x + p.y;
          }
        }
      }
      if (!SUMMARY) {
        // sum over the channel's lanes; with four lanes or more the four tokens are scattered
        // over them (lane q ends with token q mod 4), with two each ends with two tokens
        const int b0 = q & 1, b1 = (q >> 1) & 1;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float r0 = __shfl_xor_sync(0xffffffffu, b0 ? pv[r][0] : pv[r][1], 1);
          const float k0 = (b0 ? pv[r][1] : pv[r][0]) + r0;  // token b0
          const float r1 = __shfl_xor_sync(0xffffffffu, b0 ? pv[r][2] : pv[r][3], 1);
          const float k1 = (b0 ? pv[r][3] : pv[r][2]) + r1;  // token 2 + b0
          float* yr = ysm + k4 * 4 * S::kY + cg * R + r;
          if constexpr (LPC == 2) {
            yr[b0 * S::kY] += k0;
            yr[(2 + b0) * S::kY] += k1;
          } else {
            const float r2 = __shfl_xor_sync(0xffffffffu, b1 ? k0 : k1, 2);
            float yq = (b1 ? k1 : k0) + r2;
#pragma unroll
            for (int o = 4; o < LPC; o <<= 1) yq += __shfl_xor_sync(0xffffffffu, yq, o);
            if (LPC == 4 || q < 4) yr[(q & 3) * S::kY] += yq;
          }
        }
      }
    }
    __syncwarp();
    if (!SUMMARY) {
#pragma unroll
      for (int i = 0; i < S::kEx; ++i) {
        const int row = et + i * kRows;
        if (eon && t + row < t1) {
          float v = ysm[row * S::kY + ec];
          if (a.z) v *= glue::silu_fast(zc[i]);
          const int64_t at = (t + row) * a.ys + d0 + ec;
          if (a.y_bf16) static_cast<__nv_bfloat16*>(a.y)[at] = __float2bfloat16_rn(v);
          else static_cast<float*>(a.y)[at] = v;
        }
      }
      __syncwarp();
    }
    if (t + TK < t1) stage(t + TK);
    __syncwarp();
  }

  // the state after the unit
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int c = cg * R + r;
    if (c >= nch) continue;
    float* to = nullptr;
    if (SUMMARY) {
      to = a.ws_state + (int64_t(unit) * a.dim + d0 + c) * N;
      if (q == 0) a.ws_dt[int64_t(unit) * a.dim + d0 + c] = sdt[r];
    } else if (last && a.state && !(s0 == s1 && resume)) {
      to = a.state + (slot * a.dim + d0 + c) * N;
    }
    if (!to) continue;
    const float hv[4] = {h01[r].x, h01[r].y, h23[r].x, h23[r].y};
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (q * 4 + k < N) to[q * 4 + k] = hv[k];
  }
}

// One token of each sequence.  LPC lanes per channel with 4 states each, a warp on 32 / LPC
// neighbouring channels (one contiguous run of the state), RB rows per CTA so that the rates
// A are read once for them and RB state loads are in flight.
template <int LPC, int RB, bool VEC>
__global__ void __launch_bounds__(128) selective_step_kernel(const SelArgs a) {
  const int lane = threadIdx.x & 31;
  const int q = lane % LPC;
  const int d = int(blockIdx.y) * (128 / LPC) + threadIdx.x / LPC;
  const int N = a.dstate, n0 = q * 4;
  const bool on = d < a.dim;
  const int g = on ? d / (a.dim / a.ngroups) : 0;
  const int64_t row0 = int64_t(blockIdx.x) * RB;
  const int64_t batch = a.ntok;

  int64_t slot[RB];
  float h[RB][4];
#pragma unroll
  for (int r = 0; r < RB; ++r) {
    slot[r] = row0 + r < batch ? warp_slot(a.slots, row0 + r, a.nslots) : -1;
    const float* p = a.state + (slot[r] * a.dim + d) * N + n0;
    const bool ok = on && slot[r] >= 0;
    if constexpr (VEC) {
      const float4 v = ok && n0 < N ? *reinterpret_cast<const float4*>(p)
                                    : make_float4(0.f, 0.f, 0.f, 0.f);
      h[r][0] = v.x; h[r][1] = v.y; h[r][2] = v.z; h[r][3] = v.w;
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) h[r][k] = ok && n0 + k < N ? p[k] : 0.f;
    }
  }
  float av[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    av[k] = on && n0 + k < N ? rate2(a.A[int64_t(d) * N + n0 + k]) : 0.f;
  const float Dd = on && a.D ? a.D[d] : 0.f;
  const float bias = on && a.dt_bias ? a.dt_bias[d] : 0.f;
#pragma unroll
  for (int r = 0; r < RB; ++r) {
    const bool ok = on && slot[r] >= 0;
    const int64_t row = row0 + r;
    const float x = ok ? load_any(a.x, row * a.xs + d, a.io_bf16) : 0.f;
    float dt = ok ? load_any(a.dt, row * a.dts + d, a.dt_bf16) + bias : 0.f;
    if (a.softplus) dt = softplus_acc(dt);
    const float u = dt * x;
    float acc = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const bool in = ok && n0 + k < N;
      const int64_t at = int64_t(g) * N + n0 + k;
      const float bv = in ? load_any(a.B, row * a.bs + at, a.io_bf16) : 0.f;
      const float cv = in ? load_any(a.C, row * a.cs + at, a.io_bf16) : 0.f;
      h[r][k] = fmaf(ex2(dt * av[k]), h[r][k], u * bv);
      acc = fmaf(cv, h[r][k], acc);
    }
#pragma unroll
    for (int o = 1; o < LPC; o <<= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    if (ok) {
      float* p = a.state + (slot[r] * a.dim + d) * N + n0;
      if constexpr (VEC) {
        if (n0 < N)
          *reinterpret_cast<float4*>(p) = make_float4(h[r][0], h[r][1], h[r][2], h[r][3]);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (n0 + k < N) p[k] = h[r][k];
      }
      if (q == 0) {
        float v = fmaf(Dd, x, acc);
        if (a.z) v *= glue::silu_fast(load_any(a.z, row * a.zs + d, a.io_bf16));
        if (a.y_bf16) static_cast<__nv_bfloat16*>(a.y)[row * a.ys + d] = __float2bfloat16_rn(v);
        else static_cast<float*>(a.y)[row * a.ys + d] = v;
      }
    }
  }
}

}  // namespace cache
}  // namespace ssd
