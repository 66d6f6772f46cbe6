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
#include <limits.h>

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
  bool io_bf16, dt_bf16, y_bf16, softplus;
  bool by_length;  // whole sequences only, at most kSorted: the longest come first
};

// Decay rates in log2 units; a rate of -inf is held finite, so that an identity step (dt = 0)
// leaves the state and does not make a NaN of it.
__device__ __forceinline__ float rate2(float a) {
  const float r = a * kLog2e;
  return r < -1e38f ? -1e38f : r;
}

// softplus(v) = max(v, 0) + log(1 + e), e = e^-|v| in (0, 1]: no exponential overflows.  log(1 + e) =
// e p(e) keeps the relative accuracy of small results; p is the Chebyshev interpolant of degree 9
// of log(1 + e) / e on [0, 1] (off by 5e-9; with its float32 arithmetic by 1.3e-7).
__device__ __forceinline__ constexpr float log1p_coef(int k) {
  constexpr float c[10] = {1.f,           -0.499998927f, 0.333297104f,  -0.249516159f,
                           0.196632743f,  -0.152696669f, 0.105436236f,  -0.0563736111f,
                           0.0195425265f, -0.00317605701f};
  return c[k];
}
__device__ __forceinline__ float softplus_acc(float v) {
  const float e = ex2(-fabsf(v) * kLog2e);
  float p = log1p_coef(9);
#pragma unroll
  for (int k = 8; k >= 0; --k) p = fmaf(p, e, log1p_coef(k));
  return fmaf(p, e, fmaxf(v, 0.f));
}
// Two warps scan one unit: a sequence (chunk == 0) or a chunk of one, for 32 / LPC channels of
// one group; LPC lanes per channel hold SPL of its states each.  SUMMARY: only the state after
// the chunk, from zero (or, for a sequence's first chunk, from the sequence's initial state), and
// the chunk's sum of dt; those give the scan of a later chunk its entering state,
// h <- exp(A sum_dt) h + S chunk by chunk.
//
// Tokens come in stages of 16.  One warp steps through a stage's tokens; meanwhile the other
// prepares the next stage (converts the loaded values, softplus, dt x, D x, into shared memory),
// loads the one after it into registers, and finishes the stage before (adds the lanes' sums,
// gate, output).  They meet at one barrier a stage.  Done by one warp, one after the other, the
// preparation costs a third of the time wherever a scheduler has a single sequence to work on.
// VEC: a lane loads EX neighbouring channels of one row (and EB neighbouring states) in one
// access, which asks for rows of 16-byte multiples; else neighbouring lanes load neighbouring
// channels one by one.  Nothing branches between a load and its use, and addresses are a pointer
// per input that moves on by a stage.
// Why two lanes per channel for 16 states: reading B and C fills registers at 128 bytes a clock
// and SM, or 256 where a warp reads one or two addresses, and every lane reads its states' B and
// C anew; with four lanes of four states that takes longer than the exponentials.
// Measured, 5120 bf16 channels, 16 states, softplus and gate: four prompts of 2300 to 5000 tokens in
// 528 us, 71% of the ex2 rate; ragged ones are bound by the longest, at 77 ns a token (709 us where it
// has 9140 of 16384).  One prompt of 16384 tokens and 1536 channels, in chunks: 283.5 us.
constexpr int kStage = 16;

// The sequence that `rank` others come before, by falling length; nseq <= kSorted.  Call with the
// whole warp.
constexpr int kSorted = 128;
__device__ __forceinline__ int seq_of_rank(const int* __restrict__ cu, int nseq, int rank) {
  constexpr int M = kSorted / 32;
  const int lane = threadIdx.x & 31;
  int len[M], before[M];
#pragma unroll
  for (int m = 0; m < M; ++m) {
    const int i = m * 32 + lane;
    len[m] = i < nseq ? cu[i + 1] - cu[i] : INT_MIN;
    before[m] = 0;
  }
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll 1
    for (int e = 0; e < 32 && m * 32 + e < nseq; ++e) {
      const int l = __shfl_sync(0xffffffffu, len[m], e), j = m * 32 + e;
#pragma unroll
      for (int k = 0; k < M; ++k)
        before[k] += l > len[k] || (l == len[k] && j < k * 32 + lane);
    }
  int found = 0;
#pragma unroll
  for (int m = 0; m < M; ++m) {
    const unsigned hit = __ballot_sync(0xffffffffu, m * 32 + lane < nseq && before[m] == rank);
    if (hit) found = m * 32 + __ffs(hit) - 1;
  }
  return found;
}

template <typename T, typename TD, int LPC, int SPL, bool VEC, bool SUMMARY>
__global__ void __launch_bounds__(64, 8) selective_varlen_kernel(const SelArgs a) {
  constexpr int CH = 32 / LPC;         // channels of the unit
  constexpr int NP = LPC * SPL;        // states, padded
  constexpr int EX = CH / 2;           // x, dt, z elements per lane and stage
  constexpr int EB = NP / 2;           // B, C elements per lane and stage
  constexpr int P = SPL / 2;           // pairs of states
  constexpr int RX = VEC ? 0 : 32 / CH;  // rows between a lane's elements
  constexpr int RB = VEC ? 0 : (NP >= 32 ? 1 : 32 / NP);
  constexpr int CB = NP / 32 > 1 ? NP / 32 : 1;  // B, C elements of a row per lane
  // two stages each; arrays of their own, so that the compiler may move loads of one over stores
  // to another
  __shared__ __align__(16) float2 du[2][kStage * CH];
  __shared__ __align__(16) float bsm[2][kStage * NP], csm[2][SUMMARY ? 4 : kStage * NP];
  __shared__ __align__(16) float ysm[2][SUMMARY ? 4 : kStage * 32];
  using RawX = Raw<T, EX, VEC>;
  using RawD = Raw<TD, EX, VEC>;
  using RawB = Raw<T, EB, VEC>;
  // Wide loads of bf16 rows go through a ring in shared memory, kRing stages deep (four prompts at
  // 5120 channels, the longest of 9140 tokens: 840 -> 724 us; of 5020: 565 -> 536).  Float32 rows fill
  // twice the ring and the copies' time: 317 -> 351 us even, 36 -> 42 us for 33 short ones; they go
  // into registers.
  constexpr bool RING = VEC && sizeof(T) == 2;
  constexpr int kRing = 2;
  constexpr int kSlot = RING ? 32 * (2 * RawX::kPieces + RawD::kPieces + 2 * RawB::kPieces) : 1;
  __shared__ __align__(16) uint4 ring[RING ? kRing * kSlot : 1];
  // place of channel c in the rows of token k: what lanes on the same channels of eight rows touch
  // together lies on banks of its own
  auto place = [](int k, int c) { return c ^ (k & (CH < 8 ? CH - 1 : 7)); };

  const int lane = threadIdx.x & 31;
  // Which warp steps and which prepares.  CTAs of two warps take the SM's four schedulers in fixed
  // pairs, so that "the first warp" would be on the same two in all of them; taking turns by the
  // hardware's warp slot spreads the stepping warps (and their exponentials) over all four.
  __shared__ int first_steps;
  if (threadIdx.x == 0) {
    unsigned slot_id;
    asm volatile("mov.u32 %0, %%warpid;" : "=r"(slot_id));
    first_steps = !(slot_id >> 2 & 1);
  }
  __syncthreads();
  const bool steps = (threadIdx.x < 32) == bool(first_steps);
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
  int seq = !a.chunk && a.by_length ? seq_of_rank(a.cu, a.nseq, unit) : unit;
  int chunk = 0, nchunk = 1;
  if (a.chunk) {
    seq = -1;
    int base = 0;
    bool ordered = true;
    for (int i0 = 0; i0 < a.nseq; i0 += 32) {
      const int i = i0 + lane;
      int n = 0;
      if (i < a.nseq) {
        const int s = a.cu[i], e = a.cu[i + 1];
        ordered &= s >= 0 && s <= e && e <= a.ntok;
        n = e > s ? int((min(int64_t(e) - s, a.ntok) + a.chunk - 1) / a.chunk) : 1;
      }
      int incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      const unsigned m = __ballot_sync(0xffffffffu, unit < base + incl && i < a.nseq);
      if (m && seq < 0) {
        const int l = __ffs(m) - 1;
        seq = i0 + l;
        nchunk = __shfl_sync(0xffffffffu, n, l);
        chunk = unit - (base + __shfl_sync(0xffffffffu, incl, l) - nchunk);
      }
      base = min(base + __shfl_sync(0xffffffffu, incl, 31), 1 << 30);
    }
    // bounds that fall or leave the rows can name more chunks than there is room for: with them
    // every sequence is one unit
    if (!__all_sync(0xffffffffu, ordered)) {
      seq = unit < a.nseq ? unit : -1;
      chunk = 0;
      nchunk = 1;
    }
    if (seq < 0) return;
  }
  if (SUMMARY && nchunk == 1) return;
  const int64_t s0 = a.cu[seq], s1 = a.cu[seq + 1];
  if (s0 < 0 || s1 < s0 || s1 > a.ntok) return;
  const int64_t slot = a.state || a.slots ? warp_slot(a.slots, seq, a.nslots) : 0;
  if (slot < 0) return;
  const bool last = chunk == nchunk - 1;
  const bool resume = a.state && a.resume && a.resume[seq];

  if (SUMMARY && last) return;  // no chunk after it asks
  const int64_t t0 = s0 + int64_t(chunk) * a.chunk;
  const int64_t t1 = last ? s1 : t0 + a.chunk;
  const int64_t rows = t1 - t0;
  const int64_t nst = (rows + kStage - 1) / kStage;

  if (steps) {
    // this lane's channel, states and rates
    const int q = lane % LPC, ch = lane / LPC;
    const bool con = ch < nch;
    const int d = d0 + (con ? ch : 0);
    float rate[SPL], hv[SPL];
    const float* from = nullptr;  // the state that the chunk starts from, or its first part
    if (resume && chunk == 0 && (SUMMARY || nchunk == 1)) from = a.state + (slot * a.dim + d) * N;
    // a sequence cut into chunks: its initial state was copied by the summary launch (the last
    // chunk may already have moved the slot's), the others' follow from the summaries
    const int64_t u0 = unit - chunk;
    auto summary = [&](int64_t u) { return a.ws_state + (u * a.dim + d) * N; };
    if (!SUMMARY && nchunk > 1 && (chunk > 0 || resume))
      from = summary(chunk > 0 ? u0 : u0 + nchunk - 1);
#pragma unroll
    for (int k = 0; k < SPL; ++k) {
      const int n = q * SPL + k;
      rate[k] = n < N ? rate2(a.A[int64_t(d) * N + n]) : 0.f;
      hv[k] = from && n < N ? from[n] : 0.f;
    }
    if (!SUMMARY && nchunk > 1) {
#pragma unroll 2
      for (int j = 1; j < chunk; ++j) {
        const float sum = a.ws_dt[(u0 + j) * a.dim + d];
        const float* p = summary(u0 + j);
#pragma unroll
        for (int k = 0; k < SPL; ++k) {
          const int n = q * SPL + k;
          hv[k] = fmaf(ex2(rate[k] * sum), hv[k], n < N ? p[n] : 0.f);
        }
      }
    }
    if (SUMMARY && chunk == 0 && resume && con) {
#pragma unroll
      for (int k = 0; k < SPL; ++k)
        if (q * SPL + k < N) summary(unit + nchunk - 1)[q * SPL + k] = hv[k];
    }
    float2 av[P], h[P];
#pragma unroll
    for (int m = 0; m < P; ++m) {
      av[m] = make_float2(rate[2 * m], rate[2 * m + 1]);
      h[m] = make_float2(hv[2 * m], hv[2 * m + 1]);
    }
    float sdt = 0.f;
    __syncthreads();
    for (int64_t st = 0; st < nst; ++st) {
      const int left = rows - st * kStage > kStage ? kStage : int(rows - st * kStage);
      const int buf = int(st & 1);
      const float2* pdu = du[buf];
      const float *pb = bsm[buf] + q * SPL, *pc = csm[buf] + q * SPL;
      float* py = ysm[buf];
      constexpr int kGroup = 8;  // tokens unrolled
#pragma unroll 1
      for (int k0 = 0; k0 < left; k0 += kGroup) {
        float p[kGroup];
#pragma unroll
        for (int i = 0; i < kGroup; ++i) {
          const int k = k0 + i;
          const float2 v = pdu[k * CH + place(k, ch)];
          const float2 dd = dup(v.x), uu = dup(v.y);
          float2 acc = dup(0.f);
#pragma unroll
          for (int m = 0; m < P; m += 2) {
            const float4 bv = *reinterpret_cast<const float4*>(pb + k * NP + 2 * m);
            const float2 l0 = mul2(dd, av[m]), l1 = mul2(dd, av[m + 1]);
            h[m] =
                fma2(make_float2(ex2(l0.x), ex2(l0.y)), h[m], mul2(uu, make_float2(bv.x, bv.y)));
            h[m + 1] = fma2(make_float2(ex2(l1.x), ex2(l1.y)), h[m + 1],
                            mul2(uu, make_float2(bv.z, bv.w)));
            if (!SUMMARY) {
              const float4 cv = *reinterpret_cast<const float4*>(pc + k * NP + 2 * m);
              acc = m == 0 ? mul2(make_float2(cv.x, cv.y), h[0])
                           : fma2(make_float2(cv.x, cv.y), h[m], acc);
              acc = fma2(make_float2(cv.z, cv.w), h[m + 1], acc);
            }
          }
          if (SUMMARY) sdt += v.x;
          p[i] = acc.x + acc.y;
        }
        if (!SUMMARY) {
#pragma unroll
          for (int i = 0; i < kGroup; ++i) py[(k0 + i) * 32 + place(k0 + i, ch) * LPC + q] = p[i];
        }
      }
      __syncthreads();
    }
    // the state after the unit
    if (SUMMARY && con && q == 0) a.ws_dt[int64_t(unit) * a.dim + d] = sdt;
    if (!con || (!SUMMARY && (!last || !a.state || (s0 == s1 && resume)))) return;
    float* to = SUMMARY ? a.ws_state + (int64_t(unit) * a.dim + d) * N
                        : a.state + (slot * a.dim + d) * N;
#pragma unroll
    for (int k = 0; k < SPL; ++k)
      if (q * SPL + k < N) to[q * SPL + k] = k & 1 ? h[k / 2].y : h[k / 2].x;
    return;
  }

  // the preparing warp: a lane's elements of a stage are rows row0 + i RX, channel (VEC:
  // channels) c0 on
  const bool gate = !SUMMARY && a.z;
  const int row0 = VEC ? lane / 2 : lane / CH, c0 = VEC ? lane % 2 * EX : lane % CH;
  const bool eon = c0 < nch;
  const int ec = d0 + (eon ? c0 : 0);
  const int brow0 = VEC ? lane / 2 : NP >= 32 ? 0 : lane / NP;
  const int bn = VEC ? lane % 2 * EB : NP >= 32 ? lane : lane % NP;
  const T* px = static_cast<const T*>(a.x) + t0 * a.xs + ec;
  const TD* pt = static_cast<const TD*>(a.dt) + t0 * a.dts + ec;
  const T* pz = gate ? static_cast<const T*>(a.z) + t0 * a.zs + ec : nullptr;
  const T* pb = static_cast<const T*>(a.B) + t0 * a.bs + int64_t(g) * N;
  const T* pc = static_cast<const T*>(a.C) + t0 * a.cs + int64_t(g) * N;
  auto left_of = [&](int64_t st) {
    return rows - st * kStage > kStage ? kStage : int(rows - st * kStage);
  };
  RawX rx, rz;
  RawD rd;
  RawB rb, rc;
  // D x and the gate of the two stages that are not finished
  float skip0[EX], skip1[EX], gate0[EX], gate1[EX];
  // Loads of stage st, into the ring, where the lane finds them when the stage is prepared, or into
  // registers, one stage ahead.  Rows past the end read the last one again.
  auto load = [&](int64_t st) {
    if constexpr (RING) {
      if (st < nst) {
        const int64_t r = min(row0, left_of(st) - 1);
        uint32_t to = uint32_t(__cvta_generic_to_shared(ring + (st % kRing) * kSlot + lane));
        RawX::copy(to, px + r * a.xs);
        to += 512 * RawX::kPieces;
        RawD::copy(to, pt + r * a.dts);
        to += 512 * RawD::kPieces;
        RawB::copy(to, pb + r * a.bs + bn);
        to += 512 * RawB::kPieces;
        if (!SUMMARY) RawB::copy(to, pc + r * a.cs + bn);
        to += 512 * RawB::kPieces;
        if (gate) RawX::copy(to, pz + r * a.zs);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      if (st >= nst) return;
    } else if constexpr (VEC) {
      if (st >= nst) return;
      const int64_t r = min(row0, left_of(st) - 1);
      rx.load(px + r * a.xs);
      rd.load(pt + r * a.dts);
      if (gate) rz.load(pz + r * a.zs);
      rb.load(pb + r * a.bs + bn);
      if (!SUMMARY) rc.load(pc + r * a.cs + bn);
    } else {
      if (st >= nst) return;
      const int left = left_of(st);
#pragma unroll
      for (int i = 0; i < EX; ++i) {
        const int64_t r = min(row0 + i * RX, left - 1);
        rx.load1(i, px + r * a.xs);
        rd.load1(i, pt + r * a.dts);
        if (gate) rz.load1(i, pz + r * a.zs);
      }
#pragma unroll
      for (int i = 0; i < EB; ++i) {
        const int64_t r = min(brow0 + i / CB * RB, left - 1);
        const int n = min(bn + i % CB * 32, N - 1);
        rb.load1(i, pb + r * a.bs + n);
        if (!SUMMARY) rc.load1(i, pc + r * a.cs + n);
      }
    }
    px += kStage * a.xs;
    pt += kStage * a.dts;
    if (gate) pz += kStage * a.zs;
    pb += kStage * a.bs;
    pc += kStage * a.cs;
  };
  float Dd[VEC ? EX : 1], bias[VEC ? EX : 1];
  auto prepare = [&](int64_t st) {
    const int left = left_of(st), buf = int(st & 1);
    if constexpr (RING) {  // the kRing - 1 stages after this one may still be on their way
      asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
      const uint4* from = ring + (st % kRing) * kSlot + lane;
      rx.take(from);
      from += 32 * RawX::kPieces;
      rd.take(from);
      from += 32 * RawD::kPieces;
      rb.take(from);
      from += 32 * RawB::kPieces;
      if (!SUMMARY) rc.take(from);
      from += 32 * RawB::kPieces;
      if (gate) rz.take(from);
    }
    constexpr int E2 = EX > 1 ? 2 : 1;
#pragma unroll
    for (int i = 0; i < EX; i += E2) {
      float xv[2] = {0.f, 0.f}, dv[2] = {0.f, 0.f};
#pragma unroll
      for (int e = 0; e < E2; ++e) {
        xv[e] = rx.get(i + e);
        dv[e] = rd.get(i + e) + bias[VEC ? i + e : 0];
        skip0[i + e] = skip1[i + e];
        skip1[i + e] = Dd[VEC ? i + e : 0] * xv[e];
      }
      float2 v2 = make_float2(dv[0], dv[1]);
      if (gate) {
        const float2 zz = make_float2(rz.get(i), E2 > 1 ? rz.get(i + E2 - 1) : 0.f);
        const float2 g2 = mul2(zz, sigmoid2(zz));
        gate0[i] = gate1[i];
        gate1[i] = g2.x;
        if (E2 > 1) {
          gate0[i + E2 - 1] = gate1[i + E2 - 1];
          gate1[i + E2 - 1] = g2.y;
        }
      }
      if (a.softplus) v2 = make_float2(softplus_acc(v2.x), softplus_acc(v2.y));
#pragma unroll
      for (int e = 0; e < E2; ++e) {
        // rows past the end are identity steps
        const int k = row0 + (i + e) * RX;
        const bool on = eon && k < left;
        const float v = on ? (e ? v2.y : v2.x) : 0.f;
        du[buf][k * CH + place(k, c0 + (VEC ? i + e : 0))] =
            make_float2(v, on ? v * xv[e] : 0.f);
      }
    }
    if constexpr (VEC) {
      const bool on = brow0 < left;
#pragma unroll
      for (int i = 0; i < EB; i += 4) {
        *reinterpret_cast<float4*>(bsm[buf] + lane * EB + i) =
            on ? make_float4(rb.get(i), rb.get(i + 1), rb.get(i + 2), rb.get(i + 3))
               : make_float4(0.f, 0.f, 0.f, 0.f);
        if (!SUMMARY)
          *reinterpret_cast<float4*>(csm[buf] + lane * EB + i) =
              on ? make_float4(rc.get(i), rc.get(i + 1), rc.get(i + 2), rc.get(i + 3))
                 : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    } else {
#pragma unroll
      for (int i = 0; i < EB; ++i) {
        const bool on = bn + i % CB * 32 < N && brow0 + i / CB * RB < left;
        bsm[buf][i * 32 + lane] = on ? rb.get(i) : 0.f;
        if (!SUMMARY) csm[buf][i * 32 + lane] = on ? rc.get(i) : 0.f;
      }
    }
  };
  auto finish = [&](int64_t st, const float (&skip)[EX], const float (&g)[EX]) {
    const int left = left_of(st), buf = int(st & 1);
    float v[EX];
#pragma unroll
    for (int i = 0; i < EX; ++i) {
      const int k = row0 + i * RX;
      const float* pp = ysm[buf] + k * 32 + place(k, c0 + (VEC ? i : 0)) * LPC;
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < LPC; e += LPC < 4 ? LPC : 4) {
        if constexpr (LPC == 2) {
          const float2 f = *reinterpret_cast<const float2*>(pp);
          sum = f.x + f.y;
        } else {
          const float4 f = *reinterpret_cast<const float4*>(pp + e);
          sum += (f.x + f.y) + (f.z + f.w);
        }
      }
      v[i] = skip[i] + sum;
      if (gate) v[i] *= g[i];
    }
    const int64_t yrow = (t0 + st * kStage) * a.ys;
    if constexpr (VEC) {
      if (eon && row0 < left) {
        const int64_t to = yrow + row0 * a.ys + ec;
        if (a.y_bf16) {
          uint32_t w[EX / 2];
#pragma unroll
          for (int i = 0; i < EX; i += 2) w[i / 2] = pack_bf16x2(v[i], v[i + 1]);
          __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.y) + to;
          if constexpr (EX == 8) *reinterpret_cast<uint4*>(o) = make_uint4(w[0], w[1], w[2], w[3]);
          else *reinterpret_cast<uint2*>(o) = make_uint2(w[0], w[1]);
        } else {
#pragma unroll
          for (int i = 0; i < EX; i += 4)
            *reinterpret_cast<float4*>(static_cast<float*>(a.y) + to + i) =
                make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < EX; ++i) {
        if (!eon || row0 + i * RX >= left) continue;
        const int64_t to = yrow + (row0 + i * RX) * a.ys + ec;
        if (a.y_bf16) static_cast<__nv_bfloat16*>(a.y)[to] = __float2bfloat16_rn(v[i]);
        else static_cast<float*>(a.y)[to] = v[i];
      }
    }
  };

  load(0);
  if constexpr (RING) {
#pragma unroll
    for (int st = 1; st < kRing; ++st) load(st);
  }
#pragma unroll
  for (int i = 0; i < (VEC ? EX : 1); ++i) {
    Dd[i] = !SUMMARY && eon && a.D ? a.D[ec + i] : 0.f;
    bias[i] = eon && a.dt_bias ? a.dt_bias[ec + i] : 0.f;
  }
  constexpr int kNext = RING ? kRing : 1;  // stages between a load and its preparation
  if (nst > 0) prepare(0);
  load(kNext);
  __syncthreads();
  for (int64_t st = 0; st < nst; ++st) {  // the other warp is on stage st
    if (!SUMMARY && st > 0) finish(st - 1, skip0, gate0);
    if (st + 1 < nst) prepare(st + 1);
    load(st + 1 + kNext);
    __syncthreads();
  }
  if (!SUMMARY && nst > 0) finish(nst - 1, skip1, gate1);
  if constexpr (RING) asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// One token of each sequence.  LPC lanes per channel with 4 states each, a warp on 32 / LPC
// neighbouring channels (one contiguous run of the state), RB (1 or 4) rows per CTA so that the
// rates A are read once for them and RB rows' loads are in flight: a thread's loads are issued
// before the first is used.  With four rows each lane of a channel prepares (softplus) and
// finishes (gate) a row of its own, and hands dt and dt x to the others by shuffles.  VEC: a
// lane's four states, and its values of B and C, come in one access each.
// 256 rows of 5120 channels, 16 states (184 MB) in 40 us, 4.6 TB/s; 65 us with every lane preparing
// every row (292 instructions a warp and row).  Short of HBM's rate because the states are asked for
// only after the walk over the earlier slots, which grows with the square of the rows (1024 rows: 177
// us, 4096: 1295).
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
