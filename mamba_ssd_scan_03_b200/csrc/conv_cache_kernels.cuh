// conv_cache_kernels.cuh -- the short causal depthwise convolution with SiLU of a Mamba block,
// with the history a cache keeps between calls: over a packed batch of prompts of different
// lengths, and for one token of each sequence.  "State Space Models (SSM)" (ultralytics.com
// glossary), section "Da S4 a Mamba" (the short convolution ahead of the selective SSM) and
// "Come funzionano gli SSM" (the recurrent form used during generation).
//
//   out_t[c] = silu(bias[c] + sum_{k<K} w[c,k] v_{t-K+1+k}[c])
//
// where v is the sequence's input u, preceded by its slot's history: the last K-1 inputs of what
// the slot has seen (zeros for a fresh sequence).  The history leaves as the last K-1 rows of
// (history, u), the inputs' own bits.
#pragma once
#include "glue_kernels.cuh"

namespace ssd {
namespace cache {

// Sites of the latched status word (ssd_common.cuh) that these kernels use.
constexpr unsigned kSiteSeq = 200, kSiteSlot = 201;

// 1 / x by the hardware's approximation (flush-to-zero; 0 for infinity).
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 1 / (1 + e^-v) and v times it, from the hardware's exponential and reciprocal: the denormals that
// the flushing forms drop are lost in the sum with 1, and each form costs two instructions less.
__device__ __forceinline__ float sigmoid(float v) { return rcp(1.f + ex2(-kLog2e * v)); }
__device__ __forceinline__ float silu(float v) { return v * sigmoid(v); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 dup(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 sigmoid2(float2 v) {
  const float2 t = mul2(v, dup(-kLog2e));
  const float2 e = add2(make_float2(ex2(t.x), ex2(t.y)), dup(1.f));
  return make_float2(rcp(e.x), rcp(e.y));
}

// VW neighbouring channels of a row: one access of up to 16 bytes.
template <typename T, int VW>
__device__ __forceinline__ void load_ch(const T* p, float (&v)[VW]) {
  if constexpr (VW == 1) {
    v[0] = io_traits<T>::load(p, 0);
  } else {
    static_assert(VW == 4, "one channel or four");
    io_traits<T>::load4(p, 0, v);
  }
}
template <typename T, int VW>
__device__ __forceinline__ void store_ch(T* p, const float (&v)[VW]) {
  if constexpr (VW == 1) {
    io_traits<T>::store(p, 0, v[0]);
  } else if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  } else {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
}
// The weights of VW neighbouring channels, VW * K values in a row.  VW > 1: w is 16-byte aligned
// and the channel index a multiple of VW.
template <int K, int VW>
__device__ __forceinline__ void load_w(const float* w, float (&wr)[VW][K]) {
#pragma unroll
  for (int i = 0; i < VW * K; i += VW) {
    if constexpr (VW == 4) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(w + i));
      const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) wr[(i + e) / K][(i + e) % K] = f[e];
    } else {
      wr[0][i] = __ldg(w + i);
    }
  }
}
// silu(b + sum_k w[k] win[k]) of VW channels, in float32 pairs where there are two.
template <int K, int VW, int W>
__device__ __forceinline__ void conv_silu_row(const float (&win)[W][VW], int first,
                                              const float (&wr)[VW][K], const float (&bv)[VW],
                                              float (&o)[VW]) {
  if constexpr (VW == 1) {
    float acc = bv[0];
#pragma unroll
    for (int k = 0; k < K; ++k) acc = fmaf(wr[0][k], win[first + k][0], acc);
    o[0] = silu(acc);
  } else {
#pragma unroll
    for (int j = 0; j < VW; j += 2) {
      float2 acc = make_float2(bv[j], bv[j + 1]);
#pragma unroll
      for (int k = 0; k < K; ++k)
        acc = fma2(make_float2(wr[j][k], wr[j + 1][k]),
                   make_float2(win[first + k][j], win[first + k][j + 1]), acc);
      const float2 out = mul2(acc, sigmoid2(acc));
      o[j] = out.x;
      o[j + 1] = out.y;
    }
  }
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
  // The same through shared memory: pieces of 16 (or one of 8) bytes by asynchronous copies, a
  // lane's own, 32 lanes to a piece
  static constexpr int kPieces = VEC ? (kWords + 3) / 4 : 0;
  __device__ __forceinline__ static void copy(uint32_t to, const T* p) {
    static_assert(kWords == 2 || kWords % 4 == 0, "whole pieces");
    const unsigned char* q = reinterpret_cast<const unsigned char*>(p);
    if constexpr (kWords == 2) {
      asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(q) : "memory");
    } else {
#pragma unroll
      for (int k = 0; k < kPieces; ++k)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + 512 * k),
                     "l"(q + 16 * k)
                     : "memory");
    }
  }
  __device__ __forceinline__ void take(const uint4* from) {
    if constexpr (kWords == 2) {
      const uint2 v = *reinterpret_cast<const uint2*>(from);
      w[0] = v.x; w[1] = v.y;
    } else {
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        const uint4 v = from[32 * k];
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

// A warp's answer: the slot of sequence i, or -1 where the sequence is to be left alone: a
// negative slot (padding), one past the cache, or one that an earlier sequence of the call
// names too (the last two are latched as SSD_ERR_INDEX).  Call with the whole warp.
__device__ __forceinline__ int64_t warp_slot(const int* __restrict__ slots, int64_t i,
                                             int64_t nslots) {
  if (!slots) return i;
  const int lane = threadIdx.x & 31;
  const int s = slots[i];
  if (s < 0) return -1;
  bool bad = s >= nslots;
  for (int64_t j = lane; j < i; j += 32) bad |= slots[j] == s;
  if (__any_sync(0xffffffffu, bad)) {
    if (lane == 0) latch_status(SSD_ERR_INDEX, kSiteSlot);
    return -1;
  }
  return s;
}

// The same for RB neighbouring rows from row0 on, in one walk over the earlier slots; rows past
// `batch` are left alone.  Call with the whole warp.
template <int RB>
__device__ __forceinline__ void warp_slots(const int* __restrict__ slots, int64_t row0,
                                           int64_t batch, int64_t nslots, int (&out)[RB]) {
  if (!slots) {
#pragma unroll
    for (int r = 0; r < RB; ++r) out[r] = row0 + r < batch ? int(row0 + r) : -1;
    return;
  }
  const int lane = threadIdx.x & 31;
  unsigned bad = 0;
#pragma unroll
  for (int r = 0; r < RB; ++r) {
    out[r] = row0 + r < batch ? slots[row0 + r] : -1;
    if (out[r] >= nslots) bad |= 1u << r;
#pragma unroll
    for (int e = 0; e < r; ++e)
      if (out[e] == out[r]) bad |= 1u << r;
  }
  for (int64_t j = lane; j < row0; j += 32) {
    const int s = slots[j];
#pragma unroll
    for (int r = 0; r < RB; ++r)
      if (s == out[r]) bad |= 1u << r;
  }
  bad = __reduce_or_sync(0xffffffffu, bad);
#pragma unroll
  for (int r = 0; r < RB; ++r) {
    if (out[r] < 0) {
      out[r] = -1;
    } else if (bad >> r & 1u) {
      out[r] = -1;
      if (lane == 0) latch_status(SSD_ERR_INDEX, kSiteSlot);
    }
  }
}

// cu_seqlens must not decrease and must stay inside [0, ntok]; a warp latches SSD_ERR_INDEX
// where it does not.  The kernels clip every access themselves.
__device__ __forceinline__ void warp_check_seqs(const int* __restrict__ cu, int nseq,
                                                int64_t ntok) {
  bool bad = false;
  for (int i = threadIdx.x & 31; i <= nseq; i += 32)
    bad |= cu[i] < 0 || cu[i] > ntok || (i > 0 && cu[i] < cu[i - 1]);
  if (__any_sync(0xffffffffu, bad) && (threadIdx.x & 31) == 0)
    latch_status(SSD_ERR_INDEX, kSiteSeq);
}

template <typename T>
struct ConvArgs {
  const T* u;
  const float* w;
  const float* bias;
  const int* cu;
  T* state;
  const int* slots;
  const unsigned char* resume;
  T* out;
  int64_t us, os, ntok, nslots;  // row strides of u and out in elements
  int nseq, cdim;
  int run;  // packed rows of a warp (prompts)
};

// Prompts.  One warp per (run of packed rows, 32 groups of VW channels), a thread walking
// its channels down the rows as conv_silu_kernel does: weights and the window in registers,
// STEP rows' loads in flight together.  Only where a run meets the start of a sequence does
// the window restart.  A run that holds a sequence's first row owns the sequence's first K-1
// rows even where they reach past the run (the rows that read the history), and moves the
// history on itself after reading it: no other warp touches the slot, so the update in place
// needs no second launch and no ordering between CTAs.
// Bound by HBM, as long as rows stay in flight: 16 prompts of 32768 tokens together, 5376 bf16
// channels, width 4, in 138 us, 5.1 TB/s (155 us without the next step's rows in flight; 193 us
// with eight channels a lane, whose scalar loads of the weights cost more than the rows).
template <typename T, int K, int VW, int STEP>
__global__ void __launch_bounds__(32) conv_varlen_kernel(const ConvArgs<T> a) {
  constexpr int W = K - 1 + STEP;
  const int lane = threadIdx.x;
  const unsigned ncb = (a.cdim + 32 * VW - 1) / (32 * VW);  // CTAs per run, neighbours in time
  const unsigned run = blockIdx.x / ncb, cb = blockIdx.x % ncb;
  const int c0 = int(cb * 32 + lane) * VW;
  const bool live = c0 < a.cdim;  // VW > 1 only where cdim is a multiple of VW
  const int64_t r0 = int64_t(run) * a.run;
  const int64_t r1 = r0 + a.run < a.ntok ? r0 + a.run : a.ntok;
  const T* ub = a.u + c0;
  T* ob = a.out + c0;

  if (run == 0) {
    if (cb == 0) warp_check_seqs(a.cu, a.nseq, a.ntok);
    // sequences of length zero have no first row: a fresh one (on the rows) leaves a history of zeros
    if (K > 1 && a.state) {
      for (int i0 = 0; i0 < a.nseq; i0 += 32) {
        const int i = i0 + lane;
        const bool z = i < a.nseq && a.cu[i] == a.cu[i + 1] && a.cu[i] >= 0 && a.cu[i] <= a.ntok &&
                       !(a.resume && a.resume[i]) && !(a.slots && a.slots[i] < 0);
        unsigned m = __ballot_sync(0xffffffffu, z);
        while (m) {
          const int j = i0 + __ffs(m) - 1;
          m &= m - 1;
          const int64_t s = warp_slot(a.slots, j, a.nslots);
          if (s < 0 || !live) continue;
          const float zero[VW] = {};
          for (int k = 0; k < K - 1; ++k)
            store_ch<T, VW>(a.state + (s * (K - 1) + k) * a.cdim + c0, zero);
        }
      }
    }
  }

  // the first sequence that ends after r0; with bounds that fall or leave the rows, where counting
  // says nothing, all sequences are looked at
  int seq = 0;
  bool ordered = true;
  for (int i0 = 0; i0 < a.nseq; i0 += 32) {
    const int i = i0 + lane;
    bool before = false;
    if (i < a.nseq) {
      const int s = a.cu[i], e = a.cu[i + 1];
      before = e <= r0;
      ordered &= s >= 0 && s <= e && e <= a.ntok;
    }
    seq += __popc(__ballot_sync(0xffffffffu, before));
  }
  ordered = __all_sync(0xffffffffu, ordered);
  if (!ordered) seq = 0;

  float wr[VW][K], bv[VW];
  load_w<K, VW>(a.w + int64_t(live ? c0 : 0) * K, wr);
#pragma unroll
  for (int j = 0; j < VW; ++j) bv[j] = live && a.bias ? a.bias[c0 + j] : 0.f;

  for (; seq < a.nseq; ++seq) {
    const int64_t s = a.cu[seq], e = a.cu[seq + 1];
    if (s >= r1) {
      if (ordered) break;
      continue;
    }
    if (e <= s || e <= r0 || s < 0 || e > a.ntok) continue;
    const bool head = s >= r0;  // the sequence starts in this run
    // rows of this piece: from the sequence's start, or from the run's start but not the rows
    // that belong to the run of the start; and, at a start, at least the first K-1 rows
    const int64_t b = head ? s : (s + K - 1 > r0 ? s + K - 1 : r0);
    int64_t end = e < r1 ? e : r1;
    if (head && s + K - 1 > end) end = s + K - 1 < e ? s + K - 1 : e;
    const int64_t slot = a.state || a.slots ? warp_slot(a.slots, seq, a.nslots) : 0;
    if (slot < 0 || b >= end) continue;

    float win[W][VW];
#pragma unroll
    for (int k = 0; k < K - 1; ++k)
#pragma unroll
      for (int j = 0; j < VW; ++j) win[k][j] = 0.f;
    if (live) {
      if (head) {
        if (K > 1 && a.state) {
          T* st = a.state + slot * (K - 1) * a.cdim + c0;
          if (a.resume && a.resume[seq]) {
#pragma unroll
            for (int k = 0; k < K - 1; ++k) load_ch<T, VW>(st + int64_t(k) * a.cdim, win[k]);
          }
          // the history after this sequence: row k is position len - (K-1) + k; below zero it
          // is a later row of the old history, which the ascending order has not overwritten
          const int64_t len = e - s;
#pragma unroll
          for (int k = 0; k < K - 1; ++k) {
            const int64_t pos = len - (K - 1) + k;
            float v[VW] = {};
            if (pos >= 0) load_ch<T, VW>(ub + (s + pos) * a.us, v);
            else if (a.resume && a.resume[seq])
              load_ch<T, VW>(st + (K - 1 + pos) * a.cdim, v);
            store_ch<T, VW>(st + int64_t(k) * a.cdim, v);
          }
        }
      } else {
#pragma unroll
        for (int k = 0; k < K - 1; ++k) load_ch<T, VW>(ub + (b - (K - 1) + k) * a.us, win[k]);
      }
      // a step's rows as loaded: the next step's are on their way while this one's are worked on;
      // rows past the end read the last one again, and are not written
      Raw<T, VW, VW == 4> raw[STEP];
      auto load = [&](int64_t t) {
#pragma unroll
        for (int i = 0; i < STEP; ++i) {
          const T* p = ub + (t + i < end ? t + i : end - 1) * a.us;
          if constexpr (VW == 4) raw[i].load(p);
          else raw[i].load1(0, p);
        }
      };
      load(b);
      for (int64_t t = b; t < end; t += STEP) {
#pragma unroll
        for (int i = 0; i < STEP; ++i)
#pragma unroll
          for (int j = 0; j < VW; ++j) win[K - 1 + i][j] = raw[i].get(j);
        if (t + STEP < end) load(t + STEP);
#pragma unroll
        for (int i = 0; i < STEP; ++i) {
          if (t + i < end) {
            float o[VW];
            conv_silu_row<K, VW>(win, i, wr, bv, o);
            store_ch<T, VW>(ob + (t + i) * a.os, o);
          }
        }
#pragma unroll
        for (int k = 0; k < K - 1; ++k)
#pragma unroll
          for (int j = 0; j < VW; ++j) win[k][j] = win[k + STEP][j];
      }
    }
  }
}

// One token of each sequence: a thread takes VW channels of RB rows, reads each row's K-1 history
// rows and its new one, and writes the output and the moved history.  The weights are read once
// for the RB rows.  Bound by latency: the history is asked for only after the walk over the earlier slots.
// 7.1 us for 256 rows of 5376 bf16 channels (22 MB; 26 us with one row and eight channels a thread), 21
// for 1024, 116 for 4096, where the walk grows with the square of the rows.
template <typename T, int K, int VW, int RB>
__global__ void __launch_bounds__(128) conv_step_kernel(const ConvArgs<T> a) {
  const int c0 = int(blockIdx.y * blockDim.x + threadIdx.x) * VW;
  const int64_t row0 = int64_t(blockIdx.x) * RB;
  const bool live = c0 < a.cdim;
  int slot[RB];
  float win[RB][K][VW];
#pragma unroll
  for (int r = 0; r < RB; ++r) {
    const int64_t row = row0 + r < a.ntok ? row0 + r : a.ntok - 1;
    if (live) load_ch<T, VW>(a.u + row * a.us + c0, win[r][K - 1]);
  }
  warp_slots<RB>(a.slots, row0, a.ntok, a.nslots, slot);
#pragma unroll
  for (int r = 0; r < RB; ++r) {
    if (!live || slot[r] < 0) continue;
    const T* st = a.state + int64_t(slot[r]) * (K - 1) * a.cdim + c0;
#pragma unroll
    for (int k = 0; k < K - 1; ++k) load_ch<T, VW>(st + int64_t(k) * a.cdim, win[r][k]);
  }
  if (!live) return;
  float wr[VW][K], bv[VW];
  load_w<K, VW>(a.w + int64_t(c0) * K, wr);
#pragma unroll
  for (int j = 0; j < VW; ++j) bv[j] = a.bias ? a.bias[c0 + j] : 0.f;
#pragma unroll
  for (int r = 0; r < RB; ++r) {
    if (slot[r] < 0) continue;
    float o[VW];
    conv_silu_row<K, VW>(win[r], 0, wr, bv, o);
    T* st = a.state + int64_t(slot[r]) * (K - 1) * a.cdim + c0;
#pragma unroll
    for (int k = 0; k < K - 1; ++k) store_ch<T, VW>(st + int64_t(k) * a.cdim, win[r][k + 1]);
    store_ch<T, VW>(a.out + (row0 + r) * a.os + c0, o);
  }
}

}  // namespace cache
}  // namespace ssd
