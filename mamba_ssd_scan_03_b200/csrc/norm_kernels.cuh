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
// Everything is read once and kept in registers between the statistics and the result, so HBM
// bandwidth bounds both; the mean square is taken about the mean (two passes over registers),
// never as a difference of sums.
#pragma once
#include "conv_cache_kernels.cuh"

namespace ssd {
namespace norm {

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

__device__ __forceinline__ float sigm(float v) { return __fdividef(1.f, 1.f + __expf(-v)); }

// A thread's inputs of its next rows.  VW = 8: a ring of kDepth rows in shared memory that the
// thread fills for itself with 16-byte asynchronous copies, so that the loads of later rows are in
// flight while a row is worked on, and no barrier is needed.  VW = 1: plain loads.
constexpr int kDepth = 3;  // at most; fewer where a CTA's rows are too long (NormArgs::depth)
__host__ __device__ inline int ring_vecs(const NormArgs& a) {  // 16-byte pieces of 8 channels
  return (a.y_bf16 ? 1 : 2) + (a.z ? (a.z_bf16 ? 1 : 2) : 0) + (a.dout ? (a.o_bf16 ? 1 : 2) : 0);
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
          const char* from = static_cast<const char*>(base) + at * (bf16 ? 2 : 4);
          for (int k = 0; k < (bf16 ? 1 : 2); ++k, to += blockDim.x)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                             uint32_t(__cvta_generic_to_shared(to))),
                         "l"(from + 16 * k)
                         : "memory");
        };
        copy(a.y, row * a.ys + c0 + c, a.y_bf16);
        if (a.z) copy(a.z, row * a.zs + c0 + c, a.z_bf16);
        if (a.dout) copy(a.dout, row * a.os + c0 + c, a.o_bf16);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
}
// y, z and dout of unit i of the row that the ring's oldest stage holds (zeros off the end).
template <int LANES, int NV, int VW>
__device__ __forceinline__ void norm_take(const NormArgs& a, const Place<LANES, NV, VW>& p, int c0,
                                          int64_t row, const uint4* ring, int i, float (&y)[VW],
                                          float (&z)[VW], float (&d)[VW]) {
  const int c = p.col(i);
  const bool in = p.on && row < a.rows && c < p.gs;
#pragma unroll
  for (int j = 0; j < VW; ++j) y[j] = z[j] = d[j] = 0.f;
  if (!in) return;
  if constexpr (VW == 8) {
    const uint4* from = ring + i * ring_vecs(a) * blockDim.x;
    auto take = [&](float (&v)[VW], bool bf16) {
      const uint4 u = *from;
      from += blockDim.x;
      if (bf16) {
        v[0] = bf16lo(u.x); v[1] = bf16hi(u.x); v[2] = bf16lo(u.y); v[3] = bf16hi(u.y);
        v[4] = bf16lo(u.z); v[5] = bf16hi(u.z); v[6] = bf16lo(u.w); v[7] = bf16hi(u.w);
      } else {
        const uint4 t = *from;
        from += blockDim.x;
        v[0] = __uint_as_float(u.x); v[1] = __uint_as_float(u.y);
        v[2] = __uint_as_float(u.z); v[3] = __uint_as_float(u.w);
        v[4] = __uint_as_float(t.x); v[5] = __uint_as_float(t.y);
        v[6] = __uint_as_float(t.z); v[7] = __uint_as_float(t.w);
      }
    };
    take(y, a.y_bf16);
    if (a.z) take(z, a.z_bf16);
    if (a.dout) take(d, a.o_bf16);
  } else {
    load_n<VW>(a.y, row * a.ys + c0 + c, a.y_bf16, y);
    if (a.z) load_n<VW>(a.z, row * a.zs + c0 + c, a.z_bf16, z);
    if (a.dout) load_n<VW>(a.dout, row * a.os + c0 + c, a.o_bf16, d);
  }
}
// The rows of a CTA: row(k) is handed on with its ring stage when its copies have landed.
template <int LANES, int NV, int VW, typename F>
__device__ __forceinline__ void norm_rows(const NormArgs& a, const Place<LANES, NV, VW>& p, int c0,
                                          uint4* ring, const F& each) {
  const int per = VW == 8 ? NV * ring_vecs(a) * int(blockDim.x) : 0;  // of a stage
  ring += threadIdx.x;
  int in = 0, par = 0;
  int64_t ahead = p.row;
  for (; in < a.depth - 1; ++in, ahead += p.step) norm_fill(a, p, c0, ahead, ring + in * per);
  int at = 0;
  // every team of a CTA runs the same number of rounds: the sums are collective
  for (int64_t r0 = 0; r0 < a.rows; r0 += p.step, ahead += p.step, par ^= 1) {
    norm_fill(a, p, c0, ahead, ring + in * per);
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

// Threads of a CTA: 128 in teams of lanes, at most MAXT as one team (which bounds the registers).
template <int LANES, int NV, int VW, int MAXT>
__global__ void __launch_bounds__(MAXT) group_norm_kernel(const NormArgs a) {
  extern __shared__ __align__(16) uint4 ring[];
  __shared__ float buf[2][2][1][32];
  const Place<LANES, NV, VW> p(a);
  const int c0 = p.group * p.gs;
  const float inv = 1.f / p.gs;
  float w[NV][VW], bb[NV][VW];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < VW; ++j) {
      const int c = p.col(i) + j;
      const bool in = p.on && c < p.gs;
      w[i][j] = in ? __ldg(a.w + c0 + c) : 0.f;
      bb[i][j] = in && a.b ? __ldg(a.b + c0 + c) : 0.f;
    }
  norm_rows(a, p, c0, ring, [&](int64_t row, const uint4* st, int par) {
    const bool live = p.on && row < a.rows;
    float v[NV][VW], zv[NV][VW], none[VW];
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      norm_take(a, p, c0, row, st, i, v[i], zv[i], none);
#pragma unroll
      for (int j = 0; j < VW; ++j) {
        if (a.z && a.gate_first) v[i][j] *= glue::silu_fast(zv[i][j]);
        s[0] += v[i][j];
      }
    }
    float mu = 0.f;
    if (a.center) {
      team_sum<LANES>(s, buf[par][0]);
      mu = s[0] * inv;
    }
    s[0] = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VW; ++j) {
        v[i][j] -= p.col(i) < p.gs ? mu : 0.f;
        s[0] = fmaf(v[i][j], v[i][j], s[0]);
      }
    team_sum<LANES>(s, buf[par][1]);
    const float rstd = rsqrtf(fmaf(s[0], inv, a.eps));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = p.col(i);
      if (live && c < p.gs) {
        float o[VW];
#pragma unroll
        for (int j = 0; j < VW; ++j) {
          o[j] = fmaf(v[i][j] * rstd, w[i][j], bb[i][j]);
          if (a.z && !a.gate_first) o[j] *= glue::silu_fast(zv[i][j]);
        }
        store_n<VW>(a.out, row * a.os + c0 + c, a.o_bf16, o);
      }
    }
  });
}

template <int LANES, int NV, int VW, int MAXT>
__global__ void __launch_bounds__(MAXT) group_norm_bwd_kernel(const NormArgs a) {
  extern __shared__ __align__(16) uint4 ring[];
  __shared__ float buf[2][2][3][32];
  Place<LANES, NV, VW> p(a);
  const int c0 = p.group * p.gs;
  float w[NV][VW], dw[NV][VW], db[NV][VW];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < VW; ++j) {
      const int c = p.col(i) + j;
      w[i][j] = p.on && c < p.gs ? __ldg(a.w + c0 + c) : 0.f;
      dw[i][j] = db[i][j] = 0.f;
    }
  const float inv = 1.f / p.gs;
  const bool first = a.z && a.gate_first, gate_last = a.z && !a.gate_first;
  norm_rows(a, p, c0, ring, [&](int64_t row, const uint4* st, int par) {
    const bool live = p.on && row < a.rows;
    float y[NV][VW], z[NV][VW], d[NV][VW];
#pragma unroll
    for (int i = 0; i < NV; ++i) norm_take(a, p, c0, row, st, i, y[i], z[i], d[i]);
    float mu = 0.f;
    if (a.center) {
      float s[1] = {0.f};
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VW; ++j)
          s[0] += first ? y[i][j] * glue::silu_fast(z[i][j]) : y[i][j];
      team_sum<LANES>(s, buf[par][0]);
      mu = s[0] * inv;
    }
    // sums of (v - mu)^2, dn (v - mu) and dn
    float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VW; ++j) {
        const float sg = a.z ? sigm(z[i][j]) : 0.f;
        const float v = (first ? y[i][j] * (z[i][j] * sg) : y[i][j]) -
                        (p.col(i) < p.gs ? mu : 0.f);
        const float dn = (gate_last ? d[i][j] * (z[i][j] * sg) : d[i][j]) * w[i][j];
        s[0] = fmaf(v, v, s[0]);
        s[1] = fmaf(dn, v, s[1]);
        s[2] += dn;
      }
    team_sum<LANES>(s, buf[par][1]);
    const float rstd = rsqrtf(fmaf(s[0], inv, a.eps));
    const float c1 = s[1] * rstd * inv, c2 = a.center ? s[2] * inv : 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = p.col(i);
      if (live && c < p.gs) {
        float ody[VW], odz[VW];
#pragma unroll
        for (int j = 0; j < VW; ++j) {
          const float zj = z[i][j], sg = a.z ? sigm(zj) : 0.f;
          const float silu = zj * sg, slope = sg * (1.f + zj * (1.f - sg));
          const float n = ((first ? y[i][j] * silu : y[i][j]) - mu) * rstd;
          const float doj = gate_last ? d[i][j] * silu : d[i][j];
          dw[i][j] = fmaf(doj, n, dw[i][j]);
          db[i][j] += doj;
          const float dv = rstd * (doj * w[i][j] - c2 - n * c1);
          ody[j] = first ? dv * silu : dv;
          odz[j] = first ? dv * y[i][j] * slope
                         : d[i][j] * fmaf(n, w[i][j], a.b ? a.b[c0 + c + j] : 0.f) * slope;
        }
        store_n<VW>(a.dy, row * int64_t(a.cdim) + c0 + c, false, ody);
        if (a.z) store_n<VW>(a.dz, row * int64_t(a.cdim) + c0 + c, a.z_bf16, odz);
      }
    }
  });
  // one row of partial sums per CTA; the teams of one group add theirs in turn
  const int per = a.b ? 2 : 1;
  float* to = a.part + int64_t(p.cta_row) * per * a.cdim + c0;
  if constexpr (LANES != 0) {
    constexpr int kCols = MAXT * NV * VW;
    __shared__ float acc[2][kCols];
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
                db[i][j] += acc[1][base + c];
              }
              acc[0][base + c] = dw[i][j];
              acc[1][base + c] = db[i][j];
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
        if (a.b) store_n<VW>(to + a.cdim, c, false, db[i]);
      }
    }
  }
}

// dw[c] (and db[c]): the partial sums added in a fixed order, 32 columns per CTA.
__global__ void __launch_bounds__(256) norm_sum_kernel(const float* __restrict__ part, int nparts,
                                                       int per, int cdim, float* dw, float* db) {
  __shared__ float sm[8][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + tx;
  float s = 0.f;
  if (c < cdim)
    for (int k = ty; k < nparts; k += 8)
      s += part[(int64_t(k) * per + blockIdx.y) * cdim + c];
  sm[ty][tx] = s;
  __syncthreads();
  if (ty == 0 && c < cdim) {
#pragma unroll
    for (int k = 1; k < 8; ++k) s += sm[k][tx];
    (blockIdx.y ? db : dw)[c] = s;
  }
}

}  // namespace norm
}  // namespace ssd
