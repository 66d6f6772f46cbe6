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

// softplus(v) = max(v, 0) + log(1 + e), e = e^-|v| in (0, 1]: no exponential overflows, and
// small results keep their relative accuracy: log(1 + e) = 2 atanh(w), w = e / (2 + e) <= 1/3,
// by the odd series w + w^3/3 + w^5/5 + ...; the terms past w^13 / 13 are below 2^-25 of it.
__device__ __forceinline__ float softplus_acc(float v) {
  const float e = ex2(-fabsf(v) * kLog2e);
  const float w = e * rcp(2.f + e), s = w * w;
  float p = fmaf(s, 1.f / 13.f, 1.f / 11.f);
  p = fmaf(s, p, 1.f / 9.f);
  p = fmaf(s, p, 1.f / 7.f);
  p = fmaf(s, p, 1.f / 5.f);
  p = fmaf(s, p, 1.f / 3.f);
  const float w2 = w + w;
  return fmaxf(v, 0.f) + fmaf(w2 * s, p, w2);
}

// NV neighbouring values of a row as they lie in memory (one or two wide accesses), or one value
// per word.  Loading and converting are kept apart, and nothing branches between a load and the
// stage that converts it: a value is first waited for there.
template <typename T, int NV, bool VEC>
struct Raw {
  static constexpr int kWords = VEC ? NV * int(sizeof(T)) / 4 : NV;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* p) {  // VEC
    const unsigned char* q = reinterpret_cast<const unsigned char*>(p);
    if constexpr (kWords == 2) {
      const uint2 v = *reinterpret_cast<const uint2*>(q);
      w[0] = v.x; w[1] = v.y;
    } else {
#pragma unroll
      for (int k = 0; k < kWords / 4; ++k) {
        const uint4 v = reinterpret_cast<const uint4*>(q)[k];
        w[4 * k] = v.x; w[4 * k + 1] = v.y; w[4 * k + 2] = v.z; w[4 * k + 3] = v.w;
      }
    }
  }
  __device__ __forceinline__ void load1(int i, const T* p) {  // one value per word
    if constexpr (sizeof(T) == 2) w[i] = *reinterpret_cast<const unsigned short*>(p);
    else w[i] = *reinterpret_cast<const uint32_t*>(p);
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
    else if constexpr (VEC) return (i & 1) ? bf16hi(w[i / 2]) : bf16lo(w[i / 2]);
    else return bf16lo(w[i]);
  }
};

// LPC lanes per channel, each holding 4 of its (up to 4 LPC) states; R channels per lane.
template <int LPC, int R>
struct SelShape {
  static constexpr int kCg = 32 / LPC;         // channel sets of a warp
  static constexpr int kCh = kCg * R;          // channels of a warp
  static constexpr int kNp = LPC * 4;          // states, padded
  static constexpr int kTok = LPC <= 4 ? 16 : 8;  // tokens staged together
  static constexpr int kDu = 2 * kCh;          // floats per staged row of (dt, dt x) pairs
  static constexpr int kPp = LPC < 4 ? LPC : 4;  // partial sums of y per channel
  static constexpr int kY = kPp * kCh;         // floats per row of them
  static constexpr int kEx = kTok * kCh / 32;  // x, dt, z elements per lane and stage
  static constexpr int kEb = kTok * kNp / 32;  // B, C elements per lane and stage
  static_assert(kTok * kCh % 32 == 0 && 32 % kCh == 0, "whole rows per step of the warp");
  // Place of channel c's partial sums in the row of token t, in floats.  The four-way exchange
  // with t puts what the lanes of a quarter warp read together (the same channels of four
  // rows) on banks of their own.
  static __device__ __forceinline__ int part(int t, int c) {
    if constexpr (LPC == 2) return ((c >> 1) ^ (t & 3)) * 4 + (c & 1) * 2;
    else return (c ^ (t & 3)) * 4;
  }
};

// One warp scans one unit: a sequence (chunk == 0) or a chunk of one, for kCh channels of one
// group.  SUMMARY: only the state after the chunk, from zero (or, for a sequence's first chunk,
// from the sequence's initial state), and the chunk's sum of dt; those give the scan of a later
// chunk its entering state, h <- exp(A sum_dt) h + S chunk by chunk.
//
// Inputs come in stages of kTok tokens: the next stage's loads are issued into registers ahead
// of the current stage's steps, then converted (softplus, dt x, D x) once per element into
// shared memory, where the lanes of a channel all read them.  VEC: a lane loads kEx neighbouring
// channels of one row (and kEb neighbouring states) in one access, which asks for rows of 16-byte
// multiples; else neighbouring lanes load neighbouring channels one by one.
template <typename T, typename TD, int LPC, int R, bool VEC, bool SUMMARY>
__global__ void __launch_bounds__(32) selective_varlen_kernel(const SelArgs a) {
  using S = SelShape<LPC, R>;
  constexpr int TK = S::kTok, CH = S::kCh, NP = S::kNp, EX = S::kEx, EB = S::kEb;
  // arrays of their own, so that the compiler may move a token's loads over the stores before it
  __shared__ __align__(16) float du[TK * S::kDu], bsm[TK * NP], csm[TK * NP], ysm[TK * S::kY];

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

  // staging: the rows and channels of this lane's elements of a stage's tiles
  constexpr int kLr = CH / EX;  // VEC: lanes per row
  auto row = [&](int i) { return VEC ? lane / kLr : lane / CH + i * (32 / CH); };
  auto chn = [&](int i) { return VEC ? lane % kLr * EX + i : lane % CH; };
  const bool eon = chn(0) < nch;
  float Dd[EX], bias[EX];
#pragma unroll
  for (int i = 0; i < EX; ++i) {
    Dd[i] = !SUMMARY && eon && a.D ? a.D[d0 + chn(i)] : 0.f;
    bias[i] = eon && a.dt_bias ? a.dt_bias[d0 + chn(i)] : 0.f;
  }
  const T* px = static_cast<const T*>(a.x);
  const TD* pt = static_cast<const TD*>(a.dt);
  const T* pz = static_cast<const T*>(a.z);
  const T* pb = static_cast<const T*>(a.B);
  const T* pc = static_cast<const T*>(a.C);
  Raw<T, EX, VEC> rx, rz, zc;
  Raw<TD, EX, VEC> rd;
  Raw<T, EB, VEC> rb, rc;
  float skip[EX];  // D x of the staged tokens
  // Rows past the end and channels or states past the last read the last one again, and are
  // masked where they are staged.
  auto load = [&](int64_t t) {
    if constexpr (VEC) {
      const int64_t tt = min(t + row(0), t1 - 1);
      const int c = d0 + (eon ? chn(0) : 0);
      rx.load(px + tt * a.xs + c);
      rd.load(pt + tt * a.dts + c);
      if (!SUMMARY && pz) rz.load(pz + tt * a.zs + c);
      constexpr int kLb = NP / EB;  // lanes per row of B and C
      const int64_t tb = min(t + lane / kLb, t1 - 1);
      const int n = g * N + lane % kLb * EB;
      rb.load(pb + tb * a.bs + n);
      if (!SUMMARY) rc.load(pc + tb * a.cs + n);
    } else {
#pragma unroll
      for (int i = 0; i < EX; ++i) {
        const int64_t tt = min(t + row(i), t1 - 1);
        const int c = d0 + (eon ? chn(i) : 0);
        rx.load1(i, px + tt * a.xs + c);
        rd.load1(i, pt + tt * a.dts + c);
        if (!SUMMARY && pz) rz.load1(i, pz + tt * a.zs + c);
      }
#pragma unroll
      for (int i = 0; i < EB; ++i) {
        const int e = i * 32 + lane;
        const int64_t tb = min(t + e / NP, t1 - 1);
        const int n = g * N + min(e % NP, N - 1);
        rb.load1(i, pb + tb * a.bs + n);
        if (!SUMMARY) rc.load1(i, pc + tb * a.cs + n);
      }
    }
  };
  auto stage = [&](int64_t t) {
    float xv[EX], dv[EX], bv[EB], cv[EB];
#pragma unroll
    for (int i = 0; i < EX; ++i) {
      const bool on = eon && t + row(i) < t1;  // a row past the end is an identity step
      xv[i] = on ? rx.get(i) : 0.f;
      dv[i] = rd.get(i) + bias[i];
      if (a.softplus) dv[i] = softplus_acc(dv[i]);
      if (!on) dv[i] = 0.f;
      skip[i] = Dd[i] * xv[i];
    }
    zc = rz;
#pragma unroll
    for (int i = 0; i < EB; ++i) {
      const int e = VEC ? lane * EB + i : i * 32 + lane;
      const bool on = e % NP < N && t + e / NP < t1;
      bv[i] = on ? rb.get(i) : 0.f;
      if (!SUMMARY) cv[i] = on ? rc.get(i) : 0.f;
    }
    if constexpr (VEC) {
      float4* pd = reinterpret_cast<float4*>(du + row(0) * S::kDu + 2 * chn(0));
      float4* sb = reinterpret_cast<float4*>(bsm + lane * EB);
      float4* sc = reinterpret_cast<float4*>(csm + lane * EB);
#pragma unroll
      for (int i = 0; i < EX; i += 2)
        pd[i / 2] = make_float4(dv[i], dv[i] * xv[i], dv[i + 1], dv[i + 1] * xv[i + 1]);
#pragma unroll
      for (int i = 0; i < EB; i += 4) {
        sb[i / 4] = make_float4(bv[i], bv[i + 1], bv[i + 2], bv[i + 3]);
        if (!SUMMARY) sc[i / 4] = make_float4(cv[i], cv[i + 1], cv[i + 2], cv[i + 3]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < EX; ++i) {
        *reinterpret_cast<float2*>(du + row(i) * S::kDu + 2 * chn(i)) =
            make_float2(dv[i], dv[i] * xv[i]);
      }
#pragma unroll
      for (int i = 0; i < EB; ++i) {
        bsm[i * 32 + lane] = bv[i];
        if (!SUMMARY) csm[i * 32 + lane] = cv[i];
      }
    }
  };
  auto finish = [&](int64_t t) {  // y of a stage: the gate, the output's type
    float v[EX];
#pragma unroll
    for (int i = 0; i < EX; ++i) {
      const float* pp = ysm + row(i) * S::kY + S::part(row(i), chn(i));
      if constexpr (LPC == 2) {
        const float2 f = *reinterpret_cast<const float2*>(pp);
        v[i] = skip[i] + (f.x + f.y);
      } else {
        const float4 f = *reinterpret_cast<const float4*>(pp);
        v[i] = skip[i] + ((f.x + f.y) + (f.z + f.w));
      }
      if (pz) v[i] *= silu(zc.get(i));
    }
    if constexpr (VEC) {
      if (eon && t + row(0) < t1) {
        const int64_t at = (t + row(0)) * a.ys + d0 + chn(0);
        if (a.y_bf16) {
          uint32_t* to = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.y) + at);
          if constexpr (EX == 4)
            *reinterpret_cast<uint2*>(to) =
                make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
          else
            *reinterpret_cast<uint4*>(to) =
                make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                           pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
        } else {
          float4* to = reinterpret_cast<float4*>(static_cast<float*>(a.y) + at);
#pragma unroll
          for (int i = 0; i < EX; i += 4)
            to[i / 4] = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < EX; ++i) {
        if (!eon || t + row(i) >= t1) continue;
        const int64_t at = (t + row(i)) * a.ys + d0 + chn(i);
        if (a.y_bf16) static_cast<__nv_bfloat16*>(a.y)[at] = __float2bfloat16_rn(v[i]);
        else static_cast<float*>(a.y)[at] = v[i];
      }
    }
  };

  constexpr int kGroup = 4;
  if (t0 < t1) {
    load(t0);
    stage(t0);
  }
  __syncwarp();
  for (int64_t t = t0; t < t1; t += TK) {
    if (t + TK < t1) load(t + TK);
    const int steps = t1 - t < TK ? int((t1 - t + kGroup - 1) / kGroup) : TK / kGroup;
    // kGroup tokens at a time, the next ones' operands on their way while these are worked on
    float4 bn[kGroup], cn[kGroup];
    float2 dn[kGroup][R];
    auto fetch = [&](int k0) {
#pragma unroll
      for (int i = 0; i < kGroup; ++i) {
        bn[i] = *reinterpret_cast<const float4*>(bsm + (k0 + i) * NP + q * 4);
        if (!SUMMARY) cn[i] = *reinterpret_cast<const float4*>(csm + (k0 + i) * NP + q * 4);
#pragma unroll
        for (int r = 0; r < R; ++r)
          dn[i][r] =
              *reinterpret_cast<const float2*>(du + (k0 + i) * S::kDu + 2 * (cg * R + r));
      }
    };
    fetch(0);
    for (int k4 = 0; k4 < steps; ++k4) {
      float4 bv[kGroup], cv[kGroup];
      float2 dv[kGroup][R];
#pragma unroll
      for (int i = 0; i < kGroup; ++i) {
        bv[i] = bn[i];
        if (!SUMMARY) cv[i] = cn[i];
#pragma unroll
        for (int r = 0; r < R; ++r) dv[i][r] = dn[i][r];
      }
      if (k4 + 1 < steps) fetch((k4 + 1) * kGroup);
      float pv[kGroup][R];
#pragma unroll
      for (int i = 0; i < kGroup; ++i) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float2 dd = make_float2(dv[i][r].x, dv[i][r].x);
          const float2 uu = make_float2(dv[i][r].y, dv[i][r].y);
          const float2 l01 = mul2(dd, a01[r]), l23 = mul2(dd, a23[r]);
          h01[r] = fma2(make_float2(ex2(l01.x), ex2(l01.y)), h01[r],
                        mul2(uu, make_float2(bv[i].x, bv[i].y)));
          h23[r] = fma2(make_float2(ex2(l23.x), ex2(l23.y)), h23[r],
                        mul2(uu, make_float2(bv[i].z, bv[i].w)));
          if (SUMMARY) {
            sdt[r] += dd.x;
          } else {
            const float2 p2 = fma2(make_float2(cv[i].z, cv[i].w), h23[r],
                                   mul2(make_float2(cv[i].x, cv[i].y), h01[r]));
            pv[i][r] = p2.x + p2.y;
          }
        }
      }
      if (!SUMMARY) {
#pragma unroll
        for (int i = 0; i < kGroup; ++i)
#pragma unroll
          for (int r = 0; r < R; ++r) {
            float p = pv[i][r];
#pragma unroll
            for (int o = 4; o < LPC; o <<= 1) p += __shfl_xor_sync(0xffffffffu, p, o);
            // the lanes' sums meet in shared memory, added when the stage's y is finished
            if (LPC <= 4 || q < 4)
              ysm[(k4 * kGroup + i) * S::kY + S::part(i, cg * R + r) + q] = p;
          }
      }
    }
    __syncwarp();
    if (!SUMMARY) {
      finish(t);
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
// neighbouring channels (one contiguous run of the state), RB (1 or 4) rows per CTA so that the
// rates A are read once for them and RB rows' loads are in flight: a thread's loads are issued
// before the first is used.  With four rows each lane of a channel prepares (softplus) and
// finishes (gate) a row of its own, and hands dt and dt x to the others by shuffles.  VEC: a
// lane's four states, and its values of B and C, come in one access each.
template <typename T, typename TD, int LPC, int RB, bool VEC>
__global__ void __launch_bounds__(128) selective_step_kernel(const SelArgs a) {
  constexpr int OWN = RB == 4 && LPC == 2 ? 2 : 1;  // rows a lane prepares and finishes
  const int lane = threadIdx.x & 31;
  const int q = lane % LPC;
  const int d = int(blockIdx.y) * (128 / LPC) + threadIdx.x / LPC;
  const int N = a.dstate, n0 = q * 4;
  const bool on = d < a.dim && n0 < N;
  const int dc = d < a.dim ? d : 0;  // lanes off the end read channel 0 and write nothing
  const int64_t bc = int64_t(dc / (a.dim / a.ngroups)) * N + (on ? n0 : 0);
  const int64_t row0 = int64_t(blockIdx.x) * RB;
  const int64_t batch = a.ntok;
  auto own = [&](int i) { return RB == 1 ? 0 : (q & 3) + i * 2; };  // i-th own row
  auto clamp = [&](int r) { return row0 + r < batch ? row0 + r : batch - 1; };

  Raw<T, 4, VEC> rb[RB], rc[RB];
  Raw<T, 1, false> rx[OWN], rz[OWN];
  Raw<TD, 1, false> rd[OWN];
#pragma unroll
  for (int i = 0; i < OWN; ++i) {
    const int64_t row = clamp(own(i));
    rx[i].load1(0, static_cast<const T*>(a.x) + row * a.xs + dc);
    rd[i].load1(0, static_cast<const TD*>(a.dt) + row * a.dts + dc);
    if (a.z) rz[i].load1(0, static_cast<const T*>(a.z) + row * a.zs + dc);
  }
#pragma unroll
  for (int r = 0; r < RB; ++r) {
    const T* pb = static_cast<const T*>(a.B) + clamp(r) * a.bs + bc;
    const T* pc = static_cast<const T*>(a.C) + clamp(r) * a.cs + bc;
    if constexpr (VEC) {
      rb[r].load(pb);
      rc[r].load(pc);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        rb[r].load1(k, pb + (n0 + k < N ? k : 0));
        rc[r].load1(k, pc + (n0 + k < N ? k : 0));
      }
    }
  }
  float av[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    av[k] = on && n0 + k < N ? a.A[int64_t(d) * N + n0 + k] : 0.f;
  const float Dd = a.D ? a.D[dc] : 0.f;
  const float bias = a.dt_bias ? a.dt_bias[dc] : 0.f;
  int slot[RB];
  warp_slots<RB>(a.slots, row0, batch, a.nslots, slot);
  float* const at = a.state + int64_t(dc) * N + (on ? n0 : 0);
  const int64_t per = int64_t(a.dim) * N;
  float h[RB][4];
#pragma unroll
  for (int r = 0; r < RB; ++r) {
    const float* p = at + (slot[r] < 0 ? 0 : slot[r]) * per;
    if constexpr (VEC) {
      const float4 v = *reinterpret_cast<const float4*>(p);
      h[r][0] = v.x; h[r][1] = v.y; h[r][2] = v.z; h[r][3] = v.w;
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) h[r][k] = p[n0 + k < N ? k : 0];
    }
  }
  float dt[OWN], u[OWN], skip[OWN];
#pragma unroll
  for (int i = 0; i < OWN; ++i) {
    const float x = rx[i].get(0);
    dt[i] = rd[i].get(0) + bias;
    if (a.softplus) dt[i] = softplus_acc(dt[i]);
    u[i] = dt[i] * x;
    skip[i] = Dd * x;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) av[k] = rate2(av[k]);
  float acc[RB];
#pragma unroll
  for (int r = 0; r < RB; ++r) {
    float dr = dt[0], ur = u[0];
    if constexpr (RB == 4) {
      const int from = (lane & ~3) | (LPC == 2 ? (lane & 2) | (r & 1) : r);
      dr = __shfl_sync(0xffffffffu, dt[LPC == 2 ? r / 2 : 0], from);
      ur = __shfl_sync(0xffffffffu, u[LPC == 2 ? r / 2 : 0], from);
    }
    acc[r] = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      h[r][k] = fmaf(ex2(dr * av[k]), h[r][k], ur * rb[r].get(k));
      if (on && (VEC || n0 + k < N)) acc[r] = fmaf(rc[r].get(k), h[r][k], acc[r]);
    }
    if (on && slot[r] >= 0) {
      float* p = at + slot[r] * per;
      if constexpr (VEC) {
        *reinterpret_cast<float4*>(p) = make_float4(h[r][0], h[r][1], h[r][2], h[r][3]);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (n0 + k < N) p[k] = h[r][k];
      }
    }
  }
  // the channel's sums: each lane ends with its own rows'
  float sum[OWN];
  if constexpr (RB == 1) {
    sum[0] = acc[0];
#pragma unroll
    for (int o = 1; o < LPC; o <<= 1) sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], o);
  } else {
    const bool b0 = q & 1, b1 = q & 2;
    const float k0 = (b0 ? acc[1] : acc[0]) +
                     __shfl_xor_sync(0xffffffffu, b0 ? acc[0] : acc[1], 1);  // row b0
    const float k1 = (b0 ? acc[3] : acc[2]) +
                     __shfl_xor_sync(0xffffffffu, b0 ? acc[2] : acc[3], 1);  // row 2 + b0
    if constexpr (LPC == 2) {
      sum[0] = k0;
      sum[1] = k1;
    } else {
      sum[0] = (b1 ? k1 : k0) + __shfl_xor_sync(0xffffffffu, b1 ? k0 : k1, 2);
#pragma unroll
      for (int o = 4; o < LPC; o <<= 1) sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], o);
    }
  }
  if (d >= a.dim || q >= RB) return;
#pragma unroll
  for (int i = 0; i < OWN; ++i) {
    bool ok = false;
#pragma unroll
    for (int r = 0; r < RB; ++r) ok |= own(i) == r && slot[r] >= 0;
    if (!ok) continue;
    float v = skip[i] + sum[i];
    if (a.z) v *= silu(rz[i].get(0));
    const int64_t to = (row0 + own(i)) * a.ys + d;
    if (a.y_bf16) static_cast<__nv_bfloat16*>(a.y)[to] = __float2bfloat16_rn(v);
    else static_cast<float*>(a.y)[to] = v;
  }
}

}  // namespace cache
}  // namespace ssd
