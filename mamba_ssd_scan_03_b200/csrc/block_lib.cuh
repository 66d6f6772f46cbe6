// block_lib.cuh -- the C ABI of a Mamba block as a server runs it and of its norm (declared in
// include/ssd.h): argument checks, plans and launches.  Part of ssd_lib.cu, included at its end.
#pragma once
#include <atomic>

#include "conv_cache_kernels.cuh"
#include "norm_kernels.cuh"
#include "selective_cache_kernels.cuh"

namespace {

// A tensor argument: its extent in bytes from the first to the last value that rows reach.
struct Arg {
  const void* p;
  size_t bytes;
};
Arg rows_arg(const void* p, int64_t rows, int64_t stride, int64_t width, size_t es) {
  return {p, rows > 0 ? size_t((rows - 1) * stride + width) * es : 0};
}
Arg flat_arg(const void* p, int64_t n, size_t es) { return {p, p && n > 0 ? size_t(n) * es : 0}; }

// Device (or managed) memory that the current device owns.  An empty tensor has no memory.
bool here(const Arg& a, int dev) {
  if (a.bytes == 0) return true;
  if (!a.p) return false;
  cudaPointerAttributes at;
  if (cudaPointerGetAttributes(&at, a.p) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  return at.type == cudaMemoryTypeManaged || (at.type == cudaMemoryTypeDevice && at.device == dev);
}
template <size_t NI, size_t NO>
bool args_ok(const Arg (&in)[NI], const Arg (&out)[NO]) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  for (const Arg& a : in)
    if (!here(a, dev)) return false;
  for (size_t i = 0; i < NO; ++i) {
    if (!here(out[i], dev)) return false;
    for (const Arg& a : in)
      if (overlaps(out[i].p, out[i].bytes, a.p, a.bytes)) return false;
    for (size_t j = 0; j < i; ++j)
      if (overlaps(out[i].p, out[i].bytes, out[j].p, out[j].bytes)) return false;
  }
  return true;
}

bool dtype_ok(int t) { return t == SSD_F32 || t == SSD_BF16; }
size_t dtype_size(int t) { return t == SSD_BF16 ? 2 : 4; }
// rows of `es`-byte elements that 16-byte accesses can walk
bool rows16(const void* p, int64_t stride, size_t es) {
  return aligned16(p) && (size_t(stride) * es) % 16 == 0;
}

// ---- convolution -----------------------------------------------------------------------------

template <typename T, int K, int VW>
void launch_conv(const ssd::cache::ConvArgs<T>& a, cudaStream_t stream) {
  const int64_t runs = std::max<int64_t>(1, (a.ntok + a.run - 1) / a.run);
  const int64_t ncb = (a.cdim + 32 * VW - 1) / (32 * VW);
  ssd::cache::conv_varlen_kernel<T, K, VW, VW == 1 ? 8 : 6>
      <<<unsigned(runs * ncb), 32, 0, stream>>>(a);
}
template <typename T, int K, int VW>
void launch_conv_step(const ssd::cache::ConvArgs<T>& a, cudaStream_t stream) {
  const unsigned ncb = unsigned((a.cdim + 128 * VW - 1) / (128 * VW));
  // two rows per thread where that still leaves every SM a few CTAs (256 rows of 5376 channels: 7.0
  // us with two rows and four channels a thread, 7.3 with two and two, 7.9 with four and two)
  if (a.ntok / 2 * ncb >= 2 * int64_t(sm_count()))
    ssd::cache::conv_step_kernel<T, K, VW, 2>
        <<<dim3(unsigned((a.ntok + 1) / 2), ncb), 128, 0, stream>>>(a);
  else
    ssd::cache::conv_step_kernel<T, K, VW, 1><<<dim3(unsigned(a.ntok), ncb), 128, 0, stream>>>(a);
}

template <typename T>
void launch_conv_k(const ssd::cache::ConvArgs<T>& a, int kwidth, bool wide, bool step,
                   cudaStream_t stream) {
#define SSD_K(KW)                                                                \
  case KW:                                                                       \
    if (step) {                                                                  \
      if constexpr (KW > 1) {                                                    \
        if (wide) launch_conv_step<T, KW, 4>(a, stream);                         \
        else launch_conv_step<T, KW, 1>(a, stream);                              \
      }                                                                          \
    } else if (wide) {                                                           \
      launch_conv<T, KW, 4>(a, stream);                                          \
    } else {                                                                     \
      launch_conv<T, KW, 1>(a, stream);                                          \
    }                                                                            \
    break;
  switch (kwidth) {
    SSD_K(1) SSD_K(2) SSD_K(3) SSD_K(4) SSD_K(5) SSD_K(6) SSD_K(7) SSD_K(8)
  }
#undef SSD_K
}

// Packed rows of a warp: 128 where that still gives every SM 32 warps (the weights and the
// window's K-1 rows are read once per run), fewer otherwise.
int conv_run(int64_t ntok, int cdim, int vw) {
  const int64_t ncb = (cdim + 32 * vw - 1) / (32 * vw);
  int run = 128;
  while (run > 16 && (ntok + run - 1) / run * ncb < 32 * int64_t(sm_count())) run /= 2;
  return run;
}

// Both forms: step (cu == NULL) has one row per sequence.
ssd_status run_conv(const void* u, int64_t us, const float* w, const float* bias,
                    const int32_t* cu, void* state, const int32_t* slots, const uint8_t* resume,
                    void* out, int64_t os, int64_t ntok, int64_t nseq, int64_t nslots, int cdim,
                    int kwidth, ssd_dtype io, bool step, cudaStream_t stream) {
  if (ntok < 0 || nseq < 0 || cdim < 1 || kwidth < (step ? 2 : 1) || kwidth > 8 ||
      !dtype_ok(io) || us < cdim || os < cdim || nslots < 0)
    return SSD_ERR_INVALID_ARG;
  const bool kept = state != nullptr;
  if (!kept && (slots || resume || step) && !(step && nseq == 0)) return SSD_ERR_INVALID_ARG;
  if (kept && kwidth == 1) return SSD_ERR_INVALID_ARG;
  if (kept && !slots && nslots < nseq) return SSD_ERR_INVALID_ARG;
  if (nslots > INT32_MAX) return SSD_ERR_INVALID_ARG;
  if (nseq == 0) return SSD_OK;
  const size_t es = dtype_size(io);
  const Arg in[] = {rows_arg(u, ntok, us, cdim, es),
                    {w, size_t(cdim) * kwidth * 4},
                    flat_arg(bias, cdim, 4),
                    step ? Arg{nullptr, 0} : Arg{cu, size_t(nseq + 1) * 4},
                    flat_arg(slots, nseq, 4),
                    flat_arg(resume, nseq, 1)};
  const Arg outs[] = {rows_arg(out, ntok, os, cdim, es),
                      flat_arg(state, nslots * (kwidth - 1) * cdim, es)};
  if (!args_ok(in, outs)) return SSD_ERR_INVALID_ARG;
  if (ntok > INT32_MAX || nseq >= INT32_MAX || (cdim + 31) / 32 > 65535)
    return SSD_ERR_UNSUPPORTED;
  // four channels at a time: 8 or 16 bytes
  const bool wide = cdim % 4 == 0 && us % 4 == 0 && os % 4 == 0 && aligned16(u) &&
                    aligned16(out) && aligned16(state) && aligned16(w);
  const int run = conv_run(ntok, cdim, wide ? 4 : 1);
  if ((ntok + run - 1) / run * ((cdim + 31) / 32) > INT32_MAX) return SSD_ERR_UNSUPPORTED;
  auto go = [&](auto* t) {
    using T = std::remove_reference_t<decltype(*t)>;
    const ssd::cache::ConvArgs<T> a{static_cast<const T*>(u), w, bias, cu,
                                    static_cast<T*>(state), slots, resume,
                                    static_cast<T*>(out), us, os, ntok, nslots, int(nseq), cdim,
                                    run};
    launch_conv_k<T>(a, kwidth, wide, step, stream);
  };
  if (io == SSD_BF16) go(static_cast<__nv_bfloat16*>(nullptr));
  else go(static_cast<float*>(nullptr));
  return launched();
}

// ---- selective scan ----------------------------------------------------------------------------

// How packed prompts are scanned: lanes per channel, and tokens per chunk (0: whole sequences).
struct SelPlan {
  int lpc;
  int chunk;
  int64_t units;
};
int64_t sel_blocks(int dim, int ngroups, int lpc) {  // warps per unit
  const int dpg = dim / ngroups, ch = 32 / lpc;
  return int64_t(ngroups) * ((dpg + ch - 1) / ch);
}

SelPlan make_sel_plan(int64_t ntok, int nseq, int dim, int dstate, int ngroups, int64_t maxlen) {
  SelPlan p;
  p.lpc = 2;
  while (p.lpc * 8 < dstate) p.lpc *= 2;
  const int64_t sched = 4 * int64_t(sm_count());  // warp schedulers
  const int64_t len = std::min(ntok, maxlen > 0 ? maxlen : (ntok + nseq - 1) / nseq);
  const int64_t warps = nseq * sel_blocks(dim, ngroups, p.lpc);
  p.chunk = 0;
  p.units = nseq;
  if (warps < sched && len >= 128) {
    // two full rounds of CTAs (eight to an SM), chunks of at least 64 tokens.  One prompt of 16384
    // tokens and 1536 channels: 301 us, 366 with a quarter as many chunks, 342 with three times as
    // many, 1020 uncut; of 8192 and 5120: 486, 614, 484 (before rows came through the ring)
    const int64_t want = std::min(4 * sched / warps, len / 64);
    if (want > 2) {
      p.chunk = int((len + want - 1) / want + 15) / 16 * 16;
      p.units = ntok / p.chunk + nseq;
    }
  }
  return p;
}
size_t sel_workspace(const SelPlan& p, int dim, int dstate) {
  if (!p.chunk) return 0;
  return align256(size_t(p.units) * dim * dstate * 4) + align256(size_t(p.units) * dim * 4);
}

// Checks the arguments both forms share.
ssd_status check_sel(const ssd_selective_args* a, const int32_t* cu, const uint8_t* resume,
                     int64_t rows, int64_t nseq, const Arg& ws) {
  if (!a) return SSD_ERR_INVALID_ARG;
  if (rows < 0 || nseq < 0 || a->dim < 1 || a->dstate < 1 || a->ngroups < 1 ||
      a->dim % a->ngroups != 0 || !dtype_ok(a->io) ||
      (a->dt_dtype != SSD_F32 && a->dt_dtype != a->io) ||
      (a->y_dtype != SSD_F32 && a->y_dtype != a->io))
    return SSD_ERR_INVALID_ARG;
  const int64_t bc = int64_t(a->ngroups) * a->dstate;
  if (a->x_stride < a->dim || a->dt_stride < a->dim || a->y_stride < a->dim ||
      (a->z && a->z_stride < a->dim) || a->b_stride < bc || a->c_stride < bc || a->nslots < 0 ||
      a->nslots > INT32_MAX)
    return SSD_ERR_INVALID_ARG;
  if (!a->state && (a->slots || resume || (!cu && nseq > 0))) return SSD_ERR_INVALID_ARG;
  if (a->state && a->nslots < (a->slots ? std::min<int64_t>(nseq, 1) : nseq))
    return SSD_ERR_INVALID_ARG;
  if (nseq == 0) return SSD_OK;
  const size_t es = dtype_size(a->io);
  const Arg in[] = {rows_arg(a->x, rows, a->x_stride, a->dim, es),
                    rows_arg(a->dt, rows, a->dt_stride, a->dim, dtype_size(a->dt_dtype)),
                    {a->A, size_t(a->dim) * a->dstate * 4},
                    rows_arg(a->B, rows, a->b_stride, bc, es),
                    rows_arg(a->C, rows, a->c_stride, bc, es),
                    flat_arg(a->D, a->dim, 4),
                    flat_arg(a->dt_bias, a->dim, 4),
                    a->z ? rows_arg(a->z, rows, a->z_stride, a->dim, es) : Arg{nullptr, 0},
                    flat_arg(a->slots, nseq, 4),
                    flat_arg(resume, nseq, 1),
                    cu ? Arg{cu, size_t(nseq + 1) * 4} : Arg{nullptr, 0}};
  const Arg out[] = {rows_arg(a->y, rows, a->y_stride, a->dim, dtype_size(a->y_dtype)),
                     flat_arg(a->state, a->nslots * a->dim * a->dstate, 4), ws};
  if (!args_ok(in, out)) return SSD_ERR_INVALID_ARG;
  if (a->dstate > 128 || rows > INT32_MAX || nseq >= INT32_MAX) return SSD_ERR_UNSUPPORTED;
  return SSD_OK;
}

ssd::cache::SelArgs sel_args(const ssd_selective_args* a) {
  ssd::cache::SelArgs k{};
  k.x = a->x; k.dt = a->dt; k.A = a->A; k.B = a->B; k.C = a->C; k.D = a->D;
  k.dt_bias = a->dt_bias; k.z = a->z; k.y = a->y; k.state = a->state; k.slots = a->slots;
  k.xs = a->x_stride; k.dts = a->dt_stride; k.bs = a->b_stride; k.cs = a->c_stride;
  k.zs = a->z_stride; k.ys = a->y_stride;
  k.nslots = a->nslots; k.dim = a->dim; k.dstate = a->dstate; k.ngroups = a->ngroups;
  k.io_bf16 = a->io == SSD_BF16; k.dt_bf16 = a->dt_dtype == SSD_BF16;
  k.y_bf16 = a->y_dtype == SSD_BF16; k.softplus = a->softplus != 0;
  return k;
}

template <typename T, typename TD, int LPC, int SPL, bool VEC>
ssd_status launch_sel(ssd::cache::SelArgs k, const SelPlan& p, cudaStream_t stream) {
  namespace cc = ssd::cache;
  const int64_t ncb = sel_blocks(k.dim, k.ngroups, LPC);
  if (p.units * ncb > INT32_MAX) return SSD_ERR_UNSUPPORTED;
  const unsigned grid = unsigned(p.units * ncb);
  // more CTAs than the GPU holds at a time (eight to an SM): the longest sequences first, so that
  // none of them starts last
  k.by_length = !k.chunk && k.nseq > 1 && k.nseq <= cc::kSorted && grid > 8u * sm_count();
  if (k.chunk) {
    cc::selective_varlen_kernel<T, TD, LPC, SPL, VEC, true><<<grid, 64, 0, stream>>>(k);
    const ssd_status st = launched();
    if (st != SSD_OK) return st;
  }
  cc::selective_varlen_kernel<T, TD, LPC, SPL, VEC, false><<<grid, 64, 0, stream>>>(k);
  return launched();
}
// Wide loads take whole rows of 8 or 16 states and channel groups that start and end on a lane's
// eight channels, all 16-byte aligned.
bool sel_wide(const ssd::cache::SelArgs& k) {
  const size_t es = k.io_bf16 ? 2 : 4, ed = k.dt_bf16 ? 2 : 4, ey = k.y_bf16 ? 2 : 4;
  return (k.dstate == 8 || k.dstate == 16) && (k.dim / k.ngroups) % 8 == 0 &&
         rows16(k.x, k.xs, es) && rows16(k.dt, k.dts, ed) && rows16(k.B, k.bs, es) &&
         rows16(k.C, k.cs, es) && (!k.z || rows16(k.z, k.zs, es)) && rows16(k.y, k.ys, ey);
}
template <typename T, typename TD>
ssd_status launch_sel_shape(const ssd::cache::SelArgs& k, const SelPlan& p, cudaStream_t stream) {
  const bool wide = sel_wide(k);
  if (k.dstate <= 8)
    return wide ? launch_sel<T, TD, 2, 4, true>(k, p, stream)
                : launch_sel<T, TD, 2, 4, false>(k, p, stream);
  switch (p.lpc) {
    case 2:
      return wide ? launch_sel<T, TD, 2, 8, true>(k, p, stream)
                  : launch_sel<T, TD, 2, 8, false>(k, p, stream);
    case 4: return launch_sel<T, TD, 4, 8, false>(k, p, stream);
    case 8: return launch_sel<T, TD, 8, 8, false>(k, p, stream);
    default: return launch_sel<T, TD, 16, 8, false>(k, p, stream);
  }
}

template <typename T, typename TD, int LPC>
ssd_status launch_sel_step(const ssd::cache::SelArgs& k, cudaStream_t stream) {
  namespace cc = ssd::cache;
  // a lane's four states, and four values of B and C, in one access each
  const size_t four = 4 * sizeof(T);
  auto in4 = [&](const void* p, int64_t stride) {
    return reinterpret_cast<uintptr_t>(p) % four == 0 && stride % 4 == 0;
  };
  const bool vec = k.dstate % 4 == 0 && aligned16(k.state) && in4(k.B, k.bs) && in4(k.C, k.cs);
  const int64_t dblk = (k.dim + 128 / LPC - 1) / (128 / LPC);
  // four rows per CTA share the rates' loads where that still leaves every SM several CTAs
  const bool four_rows = dblk * ((k.ntok + 3) / 4) >= 4 * int64_t(sm_count());
  const dim3 grid(unsigned(four_rows ? (k.ntok + 3) / 4 : k.ntok), unsigned(dblk));
  if (dblk > 65535) return SSD_ERR_UNSUPPORTED;
  if (four_rows && vec)
    cc::selective_step_kernel<T, TD, LPC, 4, true><<<grid, 128, 0, stream>>>(k);
  else if (four_rows)
    cc::selective_step_kernel<T, TD, LPC, 4, false><<<grid, 128, 0, stream>>>(k);
  else if (vec) cc::selective_step_kernel<T, TD, LPC, 1, true><<<grid, 128, 0, stream>>>(k);
  else cc::selective_step_kernel<T, TD, LPC, 1, false><<<grid, 128, 0, stream>>>(k);
  return launched();
}
template <typename T, typename TD>
ssd_status launch_sel_step_n(const ssd::cache::SelArgs& k, cudaStream_t stream) {
  if (k.dstate <= 8) return launch_sel_step<T, TD, 2>(k, stream);
  if (k.dstate <= 16) return launch_sel_step<T, TD, 4>(k, stream);
  if (k.dstate <= 32) return launch_sel_step<T, TD, 8>(k, stream);
  if (k.dstate <= 64) return launch_sel_step<T, TD, 16>(k, stream);
  return launch_sel_step<T, TD, 32>(k, stream);
}

// ---- group norm --------------------------------------------------------------------------------

// A variant of the norm kernels (LANES, NV, VW, threads) and its grid.  `vecs`: 16-byte pieces of
// input per eight channels (they set the shared memory of a CTA's ring of rows).
struct NormPlan {
  int lanes, nv, vw, threads, depth;
  size_t smem;
  int64_t cta_rows, grid;
  bool ok;
};
// Shared memory of a ring at most; with it and the fixed arrays a CTA stays below 227 KB.
constexpr size_t kNormSmem = 192 * 1024;
NormPlan make_norm_plan(int64_t rows, int cdim, int ngroups, bool wide, int vecs) {
  NormPlan p{};
  const int gs = cdim / ngroups;
  p.vw = wide ? 8 : 1;
  const int units = (gs + p.vw - 1) / p.vw;
  p.ok = true;
  if (units <= 128) {
    p.threads = 128;
    p.lanes = units <= 8 ? 8 : 32;
    p.nv = units <= 32 ? 1 : units <= 64 ? 2 : units <= 96 && wide ? 3 : 4;
    if (p.lanes == 8 && !wide) p.lanes = 32;
    if (!wide && p.nv == 2) p.nv = 4;
  } else {
    p.lanes = 0;
    p.nv = wide ? (units <= 256 ? 1 : 2) : (units <= 2048 ? 4 : 8);
    p.threads = ((units + p.nv - 1) / p.nv + 31) / 32 * 32;
    p.ok = p.threads <= 1024;
  }
  const int teams = p.lanes ? p.threads / p.lanes : 1;
  const int gpc = std::min(teams, ngroups), rpc = teams / gpc;
  const int64_t gblk = (ngroups + gpc - 1) / gpc;
  // CTAs of an SM: about 1024 threads, and what the rings leave of its shared memory.  Rows that one
  // round of CTAs takes need no ring; else as deep a ring as leaves two CTAs to an SM.
  const size_t row = wide ? size_t(p.nv) * vecs * p.threads * 16 : 0;
  auto most = [&](int depth) {
    const int64_t per_sm = std::max<int64_t>(
        1, std::min<int64_t>(1024 / p.threads, int64_t(kNormSmem / (depth * row + 4096))));
    return std::max<int64_t>(1, sm_count() * per_sm / gblk);
  };
  p.depth = 1;
  if (wide && (rows + rpc - 1) / rpc > most(1)) {
    p.depth = int(std::min<size_t>(ssd::norm::kDepth, std::max<size_t>(2, kNormSmem / 2 / row)));
    while (p.depth > 1 && p.depth * row > kNormSmem) --p.depth;
  }
  p.smem = p.depth * row;
  p.ok = p.ok && p.smem <= kNormSmem;
  p.cta_rows = std::max<int64_t>(1, std::min((rows + rpc - 1) / rpc, most(p.depth)));
  p.grid = p.cta_rows * gblk;
  return p;
}

#define SSD_NORM_VARIANTS(X)                                                                  \
  X(8, 1, 8, 128, 8) X(32, 1, 8, 128, 8) X(32, 2, 8, 128, 4) X(32, 3, 8, 128, 4)              \
  X(32, 4, 8, 128, 3)                                                                         \
  X(0, 1, 8, 256, 4) X(0, 2, 8, 320, 2) X(0, 2, 8, 512, 1) X(0, 2, 8, 1024, 1)                \
  X(32, 1, 1, 128, 8) X(32, 4, 1, 128, 8) X(0, 4, 1, 512, 2) X(0, 8, 1, 1024, 1)

// Lets a kernel use the SM's shared memory past 48 KB; done once per kernel and device.
bool allow_smem(const void* kernel, size_t bytes, std::atomic<uint64_t>* done) {
  if (bytes <= 12 * 1024) return true;  // with the fixed arrays below 48 KB
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (dev < 64 && (done->load() & bit)) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           int(kNormSmem)) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  if (dev < 64) done->fetch_or(bit);
  return true;
}

template <typename K>
ssd_status launch_norm_kernel(K kernel, const NormPlan& p, const ssd::norm::NormArgs& a,
                              cudaStream_t stream, std::atomic<uint64_t>* done) {
  if (!allow_smem(reinterpret_cast<const void*>(kernel), p.smem, done)) return SSD_ERR_CUDA;
  kernel<<<unsigned(p.grid), p.threads, p.smem, stream>>>(a);
  return launched();
}

ssd_status launch_norm(const NormPlan& p, const ssd::norm::NormArgs& a, bool bwd,
                       cudaStream_t stream) {
#define X(L, NV, VW, MAXT, MINB)                                                              \
  if (p.lanes == L && p.nv == NV && p.vw == VW && p.threads <= MAXT) {                        \
    static std::atomic<uint64_t> done[3];                                                     \
    if (!bwd)                                                                                 \
      return launch_norm_kernel(ssd::norm::group_norm_kernel<L, NV, VW, MAXT, MINB>, p, a,    \
                                stream, &done[0]);                                            \
    if (a.b)                                                                                  \
      return launch_norm_kernel(ssd::norm::group_norm_bwd_kernel<L, NV, VW, MAXT, MINB, true>, \
                                p, a, stream, &done[1]);                                      \
    return launch_norm_kernel(ssd::norm::group_norm_bwd_kernel<L, NV, VW, MAXT, MINB, false>, \
                              p, a, stream, &done[2]);                                        \
  }
  SSD_NORM_VARIANTS(X)
#undef X
  return SSD_ERR_UNSUPPORTED;
}

// Eight channels at a time: whole units in a group, and the weight, which is read in 16-byte accesses
// too (the bias is read value by value).  The rows have their own conditions.
bool norm_wide(int cdim, int ngroups, const float* weight) {
  return (cdim / ngroups) % 8 == 0 && aligned16(weight);
}
bool norm_shape_ok(int64_t rows, int cdim, int ngroups) {
  return rows >= 0 && cdim >= 1 && ngroups >= 1 && cdim % ngroups == 0;
}

}  // namespace

extern "C" {

ssd_status ssd_conv_silu_varlen(const void* u, int64_t u_stride, const float* w,
                                const float* bias, const int32_t* cu_seqlens, void* conv_state,
                                const int32_t* slots, const uint8_t* resume, void* out,
                                int64_t out_stride, int64_t ntok, int nseq, int64_t nslots,
                                int cdim, int kwidth, ssd_dtype io, cudaStream_t stream) {
  return run_conv(u, u_stride, w, bias, cu_seqlens, conv_state, slots, resume, out, out_stride,
                  ntok, nseq, nslots, cdim, kwidth, io, false, stream);
}

ssd_status ssd_conv_silu_step(void* conv_state, const void* u, int64_t u_stride, const float* w,
                              const float* bias, const int32_t* slots, void* out,
                              int64_t out_stride, int64_t batch, int64_t nslots, int cdim,
                              int kwidth, ssd_dtype io, cudaStream_t stream) {
  return run_conv(u, u_stride, w, bias, nullptr, conv_state, slots, nullptr, out, out_stride,
                  batch, batch, nslots, cdim, kwidth, io, true, stream);
}

size_t ssd_selective_varlen_workspace_size(int64_t ntok, int nseq, int dim, int dstate,
                                           int ngroups, int64_t max_seqlen) {
  if (ntok < 0 || nseq < 1 || dim < 1 || dstate < 1 || dstate > 128 || ngroups < 1 ||
      dim % ngroups != 0 || max_seqlen < 0)
    return 0;
  return sel_workspace(make_sel_plan(ntok, nseq, dim, dstate, ngroups, max_seqlen), dim, dstate);
}

ssd_status ssd_selective_scan_varlen(const ssd_selective_args* args, const int32_t* cu_seqlens,
                                     const uint8_t* resume, int64_t ntok, int nseq,
                                     int64_t max_seqlen, void* workspace,
                                     size_t workspace_bytes, cudaStream_t stream) {
  if (nseq > 0 && !cu_seqlens) return SSD_ERR_INVALID_ARG;
  if (max_seqlen < 0) return SSD_ERR_INVALID_ARG;
  SelPlan p{};
  size_t need = 0;
  if (args && ntok >= 0 && nseq > 0 && args->dim > 0 && args->dstate > 0 && args->dstate <= 128 &&
      args->ngroups > 0 && args->dim % args->ngroups == 0) {
    p = make_sel_plan(ntok, nseq, args->dim, args->dstate, args->ngroups, max_seqlen);
    need = sel_workspace(p, args->dim, args->dstate);
  }
  if (need > 0 && (!workspace || workspace_bytes < need ||
                   (reinterpret_cast<uintptr_t>(workspace) & 255u)))
    return SSD_ERR_WORKSPACE;
  const ssd_status st = check_sel(args, cu_seqlens, resume, ntok, nseq,
                                  need ? Arg{workspace, need} : Arg{nullptr, 0});
  if (st != SSD_OK || nseq == 0) return st;
  ssd::cache::SelArgs k = sel_args(args);
  k.cu = cu_seqlens;
  k.resume = resume;
  k.ntok = ntok;
  k.nseq = nseq;
  k.chunk = p.chunk;
  if (need) {
    k.ws_state = static_cast<float*>(workspace);
    k.ws_dt = reinterpret_cast<float*>(
        static_cast<char*>(workspace) + align256(size_t(p.units) * k.dim * k.dstate * 4));
  }
  if (!k.io_bf16) return launch_sel_shape<float, float>(k, p, stream);
  if (k.dt_bf16) return launch_sel_shape<__nv_bfloat16, __nv_bfloat16>(k, p, stream);
  return launch_sel_shape<__nv_bfloat16, float>(k, p, stream);
}

ssd_status ssd_selective_step(const ssd_selective_args* args, int64_t batch,
                              cudaStream_t stream) {
  const ssd_status st = check_sel(args, nullptr, nullptr, batch, batch, Arg{nullptr, 0});
  if (st != SSD_OK || batch == 0) return st;
  ssd::cache::SelArgs k = sel_args(args);
  k.ntok = batch;
  if (!k.io_bf16) return launch_sel_step_n<float, float>(k, stream);
  if (k.dt_bf16) return launch_sel_step_n<__nv_bfloat16, __nv_bfloat16>(k, stream);
  return launch_sel_step_n<__nv_bfloat16, float>(k, stream);
}

ssd_status ssd_group_norm_gate(const void* y, int64_t y_stride, const float* weight,
                               const float* bias, const void* z, int64_t z_stride, void* out,
                               int64_t out_stride, int64_t rows, int cdim, int ngroups, float eps,
                               int center, int gate_first, ssd_dtype y_dtype, ssd_dtype z_dtype,
                               ssd_dtype out_dtype, cudaStream_t stream) {
  if (!norm_shape_ok(rows, cdim, ngroups) || !dtype_ok(y_dtype) || (z && !dtype_ok(z_dtype)) ||
      !dtype_ok(out_dtype) || y_stride < cdim || (z && z_stride < cdim) || out_stride < cdim ||
      !(eps >= 0.f))
    return SSD_ERR_INVALID_ARG;
  if (rows == 0) return SSD_OK;
  const size_t ey = dtype_size(y_dtype), ez = dtype_size(z_dtype), eo = dtype_size(out_dtype);
  const bool in_place = out == y && out_stride == y_stride && out_dtype == y_dtype;
  const Arg in[] = {{weight, size_t(cdim) * 4}, flat_arg(bias, cdim, 4),
                    z ? rows_arg(z, rows, z_stride, cdim, ez) : Arg{nullptr, 0},
                    in_place ? Arg{nullptr, 0} : rows_arg(y, rows, y_stride, cdim, ey)};
  const Arg outs[] = {rows_arg(out, rows, out_stride, cdim, eo)};
  if (!args_ok(in, outs)) return SSD_ERR_INVALID_ARG;
  const bool wide = norm_wide(cdim, ngroups, weight) && rows16(y, y_stride, ey) &&
                    y_stride % 8 == 0 &&
                    (!z || (rows16(z, z_stride, ez) && z_stride % 8 == 0)) &&
                    rows16(out, out_stride, eo) && out_stride % 8 == 0;
  ssd::norm::NormArgs a{};
  a.y = y; a.z = z; a.w = weight; a.b = bias; a.out = out;
  a.ys = y_stride; a.zs = z_stride; a.os = out_stride;
  a.rows = rows; a.cdim = cdim; a.ngroups = ngroups; a.eps = eps;
  a.y_bf16 = y_dtype == SSD_BF16; a.z_bf16 = z_dtype == SSD_BF16; a.o_bf16 = out_dtype == SSD_BF16;
  a.center = center != 0; a.gate_first = gate_first != 0;
  const NormPlan p = make_norm_plan(rows, cdim, ngroups, wide, ssd::norm::ring_vecs(a));
  a.depth = p.depth;
  if (!p.ok || p.grid > INT32_MAX) return SSD_ERR_UNSUPPORTED;
  return launch_norm(p, a, false, stream);
}

size_t ssd_group_norm_gate_bwd_workspace_size(int64_t rows, int cdim, int ngroups) {
  if (!norm_shape_ok(rows, cdim, ngroups) || rows == 0) return 0;
  int64_t n = make_norm_plan(rows, cdim, ngroups, false, 0).cta_rows;
  for (int vecs = 2; vecs <= 6; ++vecs)  // whatever the types
    n = std::max(n, make_norm_plan(rows, cdim, ngroups, true, vecs).cta_rows);
  return align256(size_t(n) * 2 * cdim * 4);
}

ssd_status ssd_group_norm_gate_bwd(const void* dout, int64_t dout_stride, const void* y,
                                   int64_t y_stride, const float* weight, const float* bias,
                                   const void* z, int64_t z_stride, float* dy, void* dz,
                                   float* dweight, float* dbias, int64_t rows, int cdim,
                                   int ngroups, float eps, int center, int gate_first,
                                   ssd_dtype dout_dtype, ssd_dtype y_dtype, ssd_dtype z_dtype,
                                   void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (!norm_shape_ok(rows, cdim, ngroups) || !dtype_ok(y_dtype) || (z && !dtype_ok(z_dtype)) ||
      !dtype_ok(dout_dtype) || y_stride < cdim || (z && z_stride < cdim) || dout_stride < cdim ||
      !(eps >= 0.f) || (bias == nullptr) != (dbias == nullptr) ||
      (rows > 0 && (z == nullptr) != (dz == nullptr)))
    return SSD_ERR_INVALID_ARG;
  const size_t ey = dtype_size(y_dtype), ez = dtype_size(z_dtype), eo = dtype_size(dout_dtype);
  const size_t need = ssd_group_norm_gate_bwd_workspace_size(rows, cdim, ngroups);
  if (need > 0 && (!workspace || workspace_bytes < need ||
                   (reinterpret_cast<uintptr_t>(workspace) & 255u)))
    return SSD_ERR_WORKSPACE;
  const Arg in[] = {{weight, size_t(cdim) * 4}, flat_arg(bias, cdim, 4),
                    z ? rows_arg(z, rows, z_stride, cdim, ez) : Arg{nullptr, 0},
                    rows_arg(y, rows, y_stride, cdim, ey),
                    rows_arg(dout, rows, dout_stride, cdim, eo)};
  const Arg outs[] = {flat_arg(dy, rows * cdim, 4),
                      z ? flat_arg(dz, rows * cdim, ez) : Arg{nullptr, 0},
                      {dweight, size_t(cdim) * 4}, flat_arg(dbias, cdim, 4),
                      need ? Arg{workspace, need} : Arg{nullptr, 0}};
  if (rows > 0 && !dy) return SSD_ERR_INVALID_ARG;
  if (!args_ok(in, outs)) return SSD_ERR_INVALID_ARG;
  const bool wide = norm_wide(cdim, ngroups, weight) && rows16(y, y_stride, ey) &&
                    y_stride % 8 == 0 &&
                    (!z || (rows16(z, z_stride, ez) && z_stride % 8 == 0 && aligned16(dz))) &&
                    rows16(dout, dout_stride, eo) && dout_stride % 8 == 0 && aligned16(dy);
  ssd::norm::NormArgs a{};
  a.y = y; a.z = z; a.w = weight; a.b = bias; a.dout = dout; a.dy = dy; a.dz = dz;
  a.part = static_cast<float*>(workspace);
  a.ys = y_stride; a.zs = z_stride; a.os = dout_stride;
  a.rows = rows; a.cdim = cdim; a.ngroups = ngroups; a.eps = eps;
  a.y_bf16 = y_dtype == SSD_BF16; a.z_bf16 = z_dtype == SSD_BF16; a.o_bf16 = dout_dtype == SSD_BF16;
  a.center = center != 0; a.gate_first = gate_first != 0;
  NormPlan p = make_norm_plan(rows, cdim, ngroups, wide, ssd::norm::ring_vecs(a));
  a.depth = p.depth;
  if (!p.ok || p.grid > INT32_MAX) return SSD_ERR_UNSUPPORTED;
  if (rows == 0) {
    p.cta_rows = 0;
  } else {
    const ssd_status st = launch_norm(p, a, true, stream);
    if (st != SSD_OK) return st;
  }
  const int per = bias ? 2 : 1;
  ssd::norm::norm_sum_kernel<<<dim3(unsigned((cdim + 31) / 32), unsigned(per)),
                              32 * ssd::norm::kSumRows, 0, stream>>>(
      static_cast<const float*>(workspace), int(p.cta_rows), per, cdim, dweight, dbias);
  return launched();
}

}  // extern "C"
