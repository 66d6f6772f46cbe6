// norm_kernels.cuh -- group norm over a token's channels with a SiLU gate, channels last: the
// normalisation of a Mamba block's output next to its gate ("State Space Models (SSM)"
// (ultralytics.com glossary), section "Da S4 a Mamba": the SiLU gate; the pages give no norm, the
// formulas below define it).  Rows are tokens; the cdim channels of a row form ngroups groups:
//
//   v = y * silu(z)  (gate first)  or  y         mu = mean(v) when centred, else 0
//   n = (v - mu) * rstd,  rstd = 1 / sqrt(mean((v - mu)^2) + eps)
//   out = n * w + b  [* silu(z) when the gate comes last]
//
// and its gradients, with do = dout [* silu(z) when the gate comes last] and dn = do * w:
//
//   dv = rstd * (dn - mean(dn) [centred] - n * mean(dn * n))
//   gate first: dy = dv silu(z), dz = dv y silu'(z);  last: dy = dv, dz = dout (n w + b) silu'(z)
//   dw = sum over rows of do * n,  db = sum over rows of do
//
// Every value is read once from HBM, whose bandwidth is the floor of both.  The forward kernel keeps a
// row in registers between its statistics and its result; the backward one reads it from the ring in
// shared memory again, as its registers are scarce.  The mean square is taken about the mean (a second
// pass over the values on chip), never as a difference of sums.  At 16384 rows of 5120 channels (float32
// y, bf16 z and output) the forward kernel takes 135.5 us, 5.0 TB/s, and the backward one with its sums
// 264 us, 4.4 TB/s; both wait, at 20 warps to an SM, for shared memory and for the sum over the CTA
// that each row needs (0.45 and 0.56 instructions issued a cycle; with plain loads and scalar
// arithmetic: 267 and 642 us).
#pragma once
#include "conv_cache_kernels.cuh"

namespace ssd {
namespace norm {

using cache::dup;
using cache::sigmoid2;

struct NormArgs {
  const void* y;
  const void* z;
  const float* w;
  const float* b;
  void* out;         // forward
  const void* dout;  // backward
  float* dy;
  void* dz;
  float* part;  // backward: [nparts][1 or 2][cdim] sums of dw (and db)
  int64_t ys, zs, os;  // row strides in elements (os: of out or dout)
  int64_t rows;
  int cdim, ngroups;
  float eps;
  int depth;  // rows of the ring
  bool y_bf16, z_bf16, o_bf16, center, gate_first;
};

// VW channels from element i on (VW = 8: 16-byte accesses).
template <int VW>
__device__ __forceinline__ void load_n(const void* p, int64_t i, bool bf16, float (&v)[VW]) {
  if constexpr (VW == 8) {
    if (bf16) {
      glue::vec<__nv_bfloat16>::load(static_cast<const __nv_bfloat16*>(p) + i, v);
    } else {
      const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
      const float4 a = f[0], b = f[1];
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
  } else {
    v[0] = bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i])
                : static_cast<const float*>(p)[i];
  }
}
template <int VW>
__device__ __forceinline__ void store_n(void* p, int64_t i, bool bf16, const float (&v)[VW]) {
  if constexpr (VW == 8) {
    if (bf16) {
      glue::vec<__nv_bfloat16>::store(static_cast<__nv_bfloat16*>(p) + i, v);
    } else {
      float4* f = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
      f[0] = make_float4(v[0], v[1], v[2], v[3]);
      f[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
  } else if (bf16) {
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v[0]);
  } else {
    static_cast<float*>(p)[i] = v[0];
  }
}

// Sums over a team: LANES lanes of a warp, or (LANES = 0) the whole CTA, through a buffer of its
// own per use so that one barrier is enough.
template <int LANES, int NS>
__device__ __forceinline__ void team_sum(float (&v)[NS], float (*buf)[32]) {
  constexpr int kL = LANES ? LANES : 32;
#pragma unroll
  for (int s = 0; s < NS; ++s)
#pragma unroll
    for (int o = kL / 2; o > 0; o >>= 1) v[s] += __shfl_xor_sync(0xffffffffu, v[s], o);
  if constexpr (LANES == 0) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    if (lane == 0)
#pragma unroll
      for (int s = 0; s < NS; ++s) buf[s][warp] = v[s];
    __syncthreads();
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      v[s] = lane < nw ? buf[s][lane] : 0.f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v[s] += __shfl_xor_sync(0xffffffffu, v[s], o);
    }
  }
}

// Where a thread works.  A team takes one (row, group) at a time: NV units of VW channels per
// lane.  Teams of a CTA stand on neighbouring groups; a CTA keeps its groups and strides over
// the rows, so that w stays in registers (and, backward, the sums of dw).
template <int LANES, int NV, int VW>
struct Place {
  int lane, team, teams, lanes;
  int group, gs;
  int gpc, rpc, cta_row, sub;  // groups and rows of a CTA; its place among the rows; the team's
  int64_t row, step;           // first row, and the rows of all CTAs together
  bool on;
  __device__ __forceinline__ Place(const NormArgs& a) {
    lanes = LANES ? LANES : blockDim.x;
    lane = threadIdx.x % lanes;
    team = threadIdx.x / lanes;
    teams = blockDim.x / lanes;
    gs = a.cdim / a.ngroups;
    gpc = teams < a.ngroups ? teams : a.ngroups;
    rpc = teams / gpc;
    const int gblk = (a.ngroups + gpc - 1) / gpc;
    cta_row = int(blockIdx.x) / gblk;
    group = (int(blockIdx.x) % gblk) * gpc + team % gpc;
    sub = team / gpc;
    on = group < a.ngroups && sub < rpc;
    row = int64_t(cta_row) * rpc + sub;
    step = int64_t(gridDim.x / gblk) * rpc;
  }
  __device__ __forceinline__ int col(int i) const { return (i * lanes + lane) * VW; }
};

// A thread's inputs of its next rows.  VW = 8: a ring of kDepth rows in shared memory that the
// thread fills for itself with 16-byte asynchronous copies, so that the loads of later rows are in
// flight while a row is worked on, and no barrier is needed.  VW = 1: plain loads.
constexpr int kDepth = 3;  // at most; fewer where a CTA's rows are too long (NormArgs::depth)
__host__ __device__ inline int ring_vecs(const NormArgs& a) {  // 16-byte pieces of 8 channels
  return (a.y_bf16 ? 1 : 2) + (a.z ? (a.z_bf16 ? 1 : 2) : 0) + (a.dout ? (a.o_bf16 ? 1 : 2) : 0);
}
// Where a thread's copies of its next row come from, one running pointer per input.  The forward
// kernel keeps them (143 -> 136 us at 16384 x 5120); the backward one finds the addresses anew for
// each row, as its registers are scarce (held there, they spill others: 266 -> 301 us).
template <int NV>
struct Ahead {
  const char *y, *z, *d;
  int64_t ys, zs, ds;  // bytes to the thread's next row
  int yu, zu, du;      // bytes between its units
  template <typename Pl>
  __device__ __forceinline__ Ahead(const NormArgs& a, const Pl& p, int c0) {
    const int c = c0 + p.col(0), lanes = p.lanes * 8;
    auto at = [&](const void* base, int64_t stride, bool bf16, const char*& ptr, int64_t& step,
                  int& unit) {
      const int es = bf16 ? 2 : 4;
      ptr = static_cast<const char*>(base) + (p.row * stride + c) * es;
      step = p.step * stride * es;
      unit = lanes * es;
    };
    at(a.y, a.ys, a.y_bf16, y, ys, yu);
    if (a.z) at(a.z, a.zs, a.z_bf16, z, zs, zu);
    if (a.dout) at(a.dout, a.os, a.o_bf16, d, ds, du);
  }
  __device__ __forceinline__ void next(const NormArgs& a) {
    y += ys;
    if (a.z) z += zs;
    if (a.dout) d += ds;
  }
};
__device__ __forceinline__ void copy16(uint32_t to, const char* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
template <int LANES, int NV, int VW>
__device__ __forceinline__ void norm_fill(const NormArgs& a, const Place<LANES, NV, VW>& p,
                                          const Ahead<NV>& from, int64_t row, uint4* ring) {
  if constexpr (VW == 8) {
    if (p.on && row < a.rows) {
      uint32_t to = uint32_t(__cvta_generic_to_shared(ring));
      const uint32_t piece = blockDim.x * 16;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const bool in = p.col(i) < p.gs;
        auto copy = [&](const char* src, bool bf16) {
          if (in) copy16(to, src);
          to += piece;
          if (!bf16) {
            if (in) copy16(to, src + 16);
            to += piece;
          }
        };
        copy(from.y + i * from.yu, a.y_bf16);
        if (a.z) copy(from.z + i * from.zu, a.z_bf16);
        if (a.dout) copy(from.d + i * from.du, a.o_bf16);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
}
template <int LANES, int NV, int VW>
__device__ __forceinline__ void norm_fill(const NormArgs& a, const Place<LANES, NV, VW>& p, int c0,
                                          int64_t row, uint4* ring) {
  if constexpr (VW == 8) {
    if (p.on && row < a.rows) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = p.col(i);
        if (c >= p.gs) continue;
        uint4* to = ring + i * ring_vecs(a) * blockDim.x;
        auto copy = [&](const void* base, int64_t at, bool bf16) {
          const char* src = static_cast<const char*>(base) + at * (bf16 ? 2 : 4);
          for (int k = 0; k < (bf16 ? 1 : 2); ++k, to += blockDim.x)
            copy16(uint32_t(__cvta_generic_to_shared(to)), src + 16 * k);
        };
        copy(a.y, row * a.ys + c0 + c, a.y_bf16);
        if (a.z) copy(a.z, row * a.zs + c0 + c, a.z_bf16);
        if (a.dout) copy(a.dout, row * a.os + c0 + c, a.o_bf16);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
}
// One input of a row: where a thread finds its 16-byte pieces in the ring, or in memory.
struct Stream {
  const void* p;
  int64_t stride;
  int first;  // piece of a unit
  bool bf16;
};
template <int LANES, int NV, int VW>
struct Streams {
  Stream y, z, d;
  int per;  // pieces of a unit
  uint32_t yw[NV], zw[NV], dw[NV];  // VW = 1: a row's values as they lie in memory
  __device__ __forceinline__ explicit Streams(const NormArgs& a) {
    y = {a.y, a.ys, 0, a.y_bf16};
    z = {a.z, a.zs, y.bf16 ? 1 : 2, a.z_bf16};
    d = {a.dout, a.os, z.first + (a.z ? (a.z_bf16 ? 1 : 2) : 0), a.o_bf16};
    per = ring_vecs(a);
  }
  // VW = 1: the row's values of all inputs, loaded together ahead of the first use (4001 rows of 5 x
  // 701 channels, gradients: 200 us with each waited for on its own, 134 so)
  __device__ __forceinline__ void fetch(const Place<LANES, NV, VW>& p, int c0, int64_t row) {
    if constexpr (VW == 1) {
      auto load = [&](const Stream& s, uint32_t (&w)[NV]) {
        if (!s.p) return;
        const int64_t at = row * s.stride + c0;
        if (s.bf16) {
#pragma unroll
          for (int i = 0; i < NV; ++i)
            w[i] = static_cast<const unsigned short*>(s.p)[at + min(p.col(i), p.gs - 1)];
        } else {
#pragma unroll
          for (int i = 0; i < NV; ++i)
            w[i] = static_cast<const uint32_t*>(s.p)[at + min(p.col(i), p.gs - 1)];
        }
      };
      load(y, yw);
      load(z, zw);
      load(d, dw);
    }
  }
};
// The VW values of unit i of the row whose stage `ring` is (VW = 1: that was fetched); the caller has
// checked that the unit lies in the group and the row among the rows.
template <int VW, int NV, typename St>
__device__ __forceinline__ void norm_take(const St& in, const Stream& s, const uint32_t (&w)[NV],
                                          const uint4* ring, int i, float (&v)[VW]) {
  if constexpr (VW == 8) {
    const uint4* from = ring + (i * in.per + s.first) * int(blockDim.x);
    const uint4 u = from[0];
    if (s.bf16) {
      v[0] = bf16lo(u.x); v[1] = bf16hi(u.x); v[2] = bf16lo(u.y); v[3] = bf16hi(u.y);
      v[4] = bf16lo(u.z); v[5] = bf16hi(u.z); v[6] = bf16lo(u.w); v[7] = bf16hi(u.w);
    } else {
      const uint4 t = from[blockDim.x];
      v[0] = __uint_as_float(u.x); v[1] = __uint_as_float(u.y);
      v[2] = __uint_as_float(u.z); v[3] = __uint_as_float(u.w);
      v[4] = __uint_as_float(t.x); v[5] = __uint_as_float(t.y);
      v[6] = __uint_as_float(t.z); v[7] = __uint_as_float(t.w);
    }
  } else {
    v[0] = s.bf16 ? bf16lo(w[i]) : __uint_as_float(w[i]);
  }
}
// Pairs of values (VW = 1: one value and a zero).
template <int VW>
__device__ __forceinline__ float2 pair(const float (&v)[VW], int j) {
  if constexpr (VW == 1) return make_float2(v[0], 0.f);
  else return make_float2(v[j], v[j + 1]);
}
template <int VW>
__device__ __forceinline__ void put(float (&v)[VW], int j, float2 f) {
  v[j] = f.x;
  if constexpr (VW > 1) v[j + 1] = f.y;
}

// The rows of a CTA: row(k) is handed on with its ring stage when its copies have landed.
template <bool KEEP, int LANES, int NV, int VW, typename F>
__device__ __forceinline__ void norm_rows(const NormArgs& a, const Place<LANES, NV, VW>& p, int c0,
                                          uint4* ring, const F& each) {
  const int per = VW == 8 ? NV * ring_vecs(a) * int(blockDim.x) : 0;  // of a stage
  ring += threadIdx.x;
  int in = 0, par = 0;
  int64_t ahead = p.row;
  Ahead<NV> from(a, p, c0);
  auto fill = [&] {
    if constexpr (KEEP) {
      norm_fill(a, p, from, ahead, ring + in * per);
      from.next(a);
    } else {
      norm_fill(a, p, c0, ahead, ring + in * per);
    }
    ahead += p.step;
  };
  for (; in < a.depth - 1; ++in) fill();
  int at = 0;
  // every team of a CTA runs the same number of rounds: the sums are collective
  for (int64_t r0 = 0; r0 < a.rows; r0 += p.step, par ^= 1) {
    fill();
    in = in + 1 == a.depth ? 0 : in + 1;
    if constexpr (VW == 8) {  // all but the depth - 1 youngest rows have landed
      if (a.depth == 3) asm volatile("cp.async.wait_group 2;" ::: "memory");
      else if (a.depth == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
      else asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    each(r0 + p.row, ring + at * per, par);
    at = at + 1 == a.depth ? 0 : at + 1;
  }
  if constexpr (VW == 8) asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Threads of a CTA: 128 in teams of lanes, at most MAXT as one team; MINB CTAs to an SM (the two
// bound the registers).
template <int LANES, int NV, int VW, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) group_norm_kernel(const NormArgs a) {
  constexpr int STEP = VW == 1 ? 1 : 2;
  extern __shared__ __align__(16) uint4 ring[];
  __shared__ float buf[2][2][1][32];
  const Place<LANES, NV, VW> p(a);
  Streams<LANES, NV, VW> in(a);
  const int c0 = p.group * p.gs;
  const float inv = 1.f / p.gs;
  const bool first = a.z && a.gate_first, last = a.z && !a.gate_first;
  float w[NV][VW];
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (p.on && p.col(i) < p.gs) load_n<VW>(a.w, c0 + p.col(i), false, w[i]);
  norm_rows<true>(a, p, c0, ring, [&](int64_t row, const uint4* st, int par) {
    const bool live = p.on && row < a.rows;
    if (live) in.fetch(p, c0, row);
    float v[NV][VW];
    float2 s2 = dup(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = p.col(i);
      if (live && c < p.gs) {
        norm_take<VW>(in, in.y, in.yw, st, i, v[i]);
        if (first) {
          float z[VW];
          norm_take<VW>(in, in.z, in.zw, st, i, z);
#pragma unroll
          for (int j = 0; j < VW; j += STEP) {
            const float2 zz = pair<VW>(z, j);
            put<VW>(v[i], j, mul2(pair<VW>(v[i], j), mul2(zz, sigmoid2(zz))));
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < VW; ++j) v[i][j] = 0.f;
      }
    }
    if (a.center) {
      float s[1];
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VW; j += STEP) s2 = cache::add2(s2, pair<VW>(v[i], j));
      s[0] = s2.x + s2.y;
      team_sum<LANES>(s, buf[par][0]);
      const float mu = s[0] * inv;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (p.col(i) < p.gs)
#pragma unroll
          for (int j = 0; j < VW; ++j) v[i][j] -= mu;
      s2 = dup(0.f);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VW; j += STEP) s2 = fma2(pair<VW>(v[i], j), pair<VW>(v[i], j), s2);
    float s[1] = {s2.x + s2.y};
    team_sum<LANES>(s, buf[par][1]);
    const float2 rstd = dup(rsqrtf(fmaf(s[0], inv, a.eps)));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = p.col(i);
      if (live && c < p.gs) {
        float o[VW];
#pragma unroll
        for (int j = 0; j < VW; j += STEP)
          put<VW>(o, j, mul2(mul2(pair<VW>(v[i], j), rstd), pair<VW>(w[i], j)));
        if (a.b) {
#pragma unroll
          for (int j = 0; j < VW; ++j) o[j] += __ldg(a.b + c0 + c + j);
        }
        if (last) {
          float z[VW];
          norm_take<VW>(in, in.z, in.zw, st, i, z);
#pragma unroll
          for (int j = 0; j < VW; j += STEP) {
            const float2 zz = pair<VW>(z, j);
            put<VW>(o, j, mul2(pair<VW>(o, j), mul2(zz, sigmoid2(zz))));
          }
        }
        store_n<VW>(a.out, row * a.os + c0 + c, a.o_bf16, o);
      }
    }
  });
}

// BIAS: sums db as well.  The row's values are read from the ring again for the gradients rather
// than held in registers across the sums.
template <int LANES, int NV, int VW, int MAXT, int MINB, bool BIAS>
__global__ void __launch_bounds__(MAXT, MINB) group_norm_bwd_kernel(const NormArgs a) {
  constexpr int STEP = VW == 1 ? 1 : 2;
  extern __shared__ __align__(16) uint4 ring[];
  __shared__ float buf[2][2][3][32];
  Place<LANES, NV, VW> p(a);
  Streams<LANES, NV, VW> in(a);
  const int c0 = p.group * p.gs;
  float w[NV][VW], dw[NV][VW], db[BIAS ? NV : 1][VW];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (p.on && p.col(i) < p.gs) load_n<VW>(a.w, c0 + p.col(i), false, w[i]);
#pragma unroll
    for (int j = 0; j < VW; ++j) {
      dw[i][j] = 0.f;
      if (BIAS) db[i][j] = 0.f;
    }
  }
  const float inv = 1.f / p.gs;
  const bool first = a.z && a.gate_first, last = a.z && !a.gate_first;
  norm_rows<false>(a, p, c0, ring, [&](int64_t row, const uint4* st, int par) {
    const bool live = p.on && row < a.rows;
    if (live) in.fetch(p, c0, row);
    // v and do of a unit's pair j, as both passes need them
    float y[VW], z[VW], d[VW];
    auto take = [&](int i) {
      norm_take<VW>(in, in.y, in.yw, st, i, y);
      norm_take<VW>(in, in.d, in.dw, st, i, d);
      if (a.z) norm_take<VW>(in, in.z, in.zw, st, i, z);
    };
    float mu = 0.f;
    if (a.center) {
      float s[1] = {0.f};
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (live && p.col(i) < p.gs) {
          take(i);
#pragma unroll
          for (int j = 0; j < VW; ++j) s[0] += first ? y[j] * cache::silu(z[j]) : y[j];
        }
      team_sum<LANES>(s, buf[par][0]);
      mu = s[0] * inv;
    }
    // sums of (v - mu)^2, dn (v - mu) and dn
    float2 t0 = dup(0.f), t1 = dup(0.f), t2 = dup(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (live && p.col(i) < p.gs) {
        take(i);
#pragma unroll
        for (int j = 0; j < VW; j += STEP) {
          float2 v = pair<VW>(y, j), dn = pair<VW>(d, j);
          if (a.z) {
            const float2 zz = pair<VW>(z, j), g = mul2(zz, sigmoid2(zz));
            if (first) v = mul2(v, g);
            else dn = mul2(dn, g);
          }
          v = cache::add2(v, make_float2(-mu, VW == 1 ? 0.f : -mu));
          dn = mul2(dn, pair<VW>(w[i], j));
          t0 = fma2(v, v, t0);
          t1 = fma2(dn, v, t1);
          t2 = cache::add2(t2, dn);
        }
      }
    float s[3] = {t0.x + t0.y, t1.x + t1.y, t2.x + t2.y};
    team_sum<LANES>(s, buf[par][1]);
    const float rstd = rsqrtf(fmaf(s[0], inv, a.eps));
    const float2 r2 = dup(rstd), c1 = dup(-s[1] * rstd * inv);
    const float2 c2 = dup(a.center ? -s[2] * inv : 0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = p.col(i);
      if (live && c < p.gs) {
        take(i);
        float ody[VW], odz[VW];
#pragma unroll
        for (int j = 0; j < VW; j += STEP) {
          const float2 yy = pair<VW>(y, j), ww = pair<VW>(w[i], j);
          float2 v = yy, dd = pair<VW>(d, j), g = dup(1.f), slope = dup(0.f);
          if (a.z) {
            const float2 zz = pair<VW>(z, j), sg = sigmoid2(zz);
            g = mul2(zz, sg);
            // silu' = sg (1 + z (1 - sg)) = sg + g (1 - sg).  Not as (sg + g) - g sg: both are of the
            // gate's size, and past 2^24 the 1 between them is lost.
            slope = fma2(g, cache::add2(dup(1.f), make_float2(-sg.x, -sg.y)), sg);
            if (first) v = mul2(yy, g);
          }
          const float2 n = mul2(cache::add2(v, dup(-mu)), r2);
          if (last) {
            float2 o = mul2(n, ww);
            if (BIAS) {
              o.x += __ldg(a.b + c0 + c + j);
              if (VW > 1) o.y += __ldg(a.b + c0 + c + j + 1);
            }
            put<VW>(odz, j, mul2(mul2(dd, o), slope));
            dd = mul2(dd, g);
          }
          put<VW>(dw[i], j, fma2(dd, n, pair<VW>(dw[i], j)));
          if (BIAS) put<VW>(db[i], j, cache::add2(pair<VW>(db[i], j), dd));
          const float2 dv = mul2(r2, fma2(dd, ww, fma2(n, c1, c2)));
          put<VW>(ody, j, first ? mul2(dv, g) : dv);
          if (first) put<VW>(odz, j, mul2(mul2(dv, yy), slope));
        }
        store_n<VW>(a.dy, row * int64_t(a.cdim) + c0 + c, false, ody);
        if (a.z) store_n<VW>(a.dz, row * int64_t(a.cdim) + c0 + c, a.z_bf16, odz);
      }
    }
  });
  // one row of partial sums per CTA; the teams of one group add theirs in turn
  constexpr int per = BIAS ? 2 : 1;
  float* to = a.part + int64_t(p.cta_row) * per * a.cdim + c0;
  if constexpr (LANES != 0) {
    constexpr int kCols = MAXT * NV * VW;
    __shared__ float acc[per][kCols];
    const int base = (p.team % p.gpc) * p.gs;
    for (int k = 0; k < p.rpc; ++k) {
      if (p.on && p.sub == k) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int j = 0; j < VW; ++j) {
            const int c = p.col(i) + j;
            if (c < p.gs) {
              if (k > 0) {
                dw[i][j] += acc[0][base + c];
                if constexpr (BIAS) db[i][j] += acc[1][base + c];
              }
              acc[0][base + c] = dw[i][j];
              if constexpr (BIAS) acc[1][base + c] = db[i][j];
            }
          }
      }
      __syncthreads();
    }
    p.on = p.on && p.sub == p.rpc - 1;
  }
  if (p.on) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = p.col(i);
      if (c < p.gs) {
        store_n<VW>(to, c, false, dw[i]);
        if constexpr (BIAS) store_n<VW>(to + a.cdim, c, false, db[i]);
      }
    }
  }
}

// dw[c] (and db[c]): the partial sums added in a fixed order, 32 columns per CTA.
constexpr int kSumRows = 32;
__global__ void __launch_bounds__(32 * kSumRows) norm_sum_kernel(const float* __restrict__ part,
                                                                 int nparts, int per, int cdim,
                                                                 float* dw, float* db) {
  __shared__ float sm[kSumRows][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + tx;
  float s = 0.f;
  if (c < cdim) {
#pragma unroll 8
    for (int k = ty; k < nparts; k += kSumRows)
      s += part[(int64_t(k) * per + blockIdx.y) * cdim + c];
  }
  sm[ty][tx] = s;
  __syncthreads();
  if (ty == 0 && c < cdim) {
#pragma unroll
    for (int k = 1; k < kSumRows; ++k) s += sm[k][tx];
    (blockIdx.y ? db : dw)[c] = s;
  }
}

}  // namespace norm
}  // namespace ssd
