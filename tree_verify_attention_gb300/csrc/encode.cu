// Queries, keys and values of a projection as the attention takes them: RMS
// norm of each query and key head, the position rotation, the values carried
// along, in one pass.
//
//   y = x / sqrt(mean(x^2) + eps) * w
//   (a, b) -> (a cos t - b sin t, b cos t + a sin t),  t = pos * freq_i
//
// The kernel is bound by memory (each element is read once and written once)
// and by latency for a few rows. A head is D / 16 lanes of a warp, each with
// two chunks of eight elements, picked so that both elements of a rotated pair
// are in one lane; the same lane then has the same eight pairs in every head
// of the row, so their sines and cosines are computed once per row and stay in
// registers. A warp works through the heads of a row; few rows are split over
// more warps.
//
// Angles: pos * freq in 32 bits would be off by 2^-8 rad at position 131072.
// The table holds turns per position as a 64-bit binary fraction, so the
// integer product pos * turns, modulo 2^64, is the angle's fraction of a turn,
// exact for the table's entry; one rounded to the nearest 2^-64 adds |pos| * 2^-65.
// The upper 32 bits go to sincospi, as 24: 2^-32 and 2^-26 of a turn.

#include "common.cuh"

namespace dfv {

// CTAs of one warp: the SM takes the next row as soon as one is done (16411 rows
// of 32 / 8 heads of 128: 75 us, by four warps 78).
constexpr int kEncWarps = 1;

struct EncodeParams {
  int n_rows, hq, hkv, rot;
  int iters, it_k, it_v;   // of a row, the key heads' and the value heads' first
  int splits, per_split;
  const void *q, *k, *v;
  int64_t q_row, q_head, k_row, k_head, v_row, v_head;
  const float *q_weight, *k_weight;
  float eps;
  const uint64_t* turns;
  const int32_t *positions, *parent, *ctx_len, *dropped;
  void *q_out, *k_out, *v_out;
  uint32_t* status;
};

// Eight consecutive elements as float32.
template <typename T, bool kVec> struct EncLoad;
template <> struct EncLoad<__nv_bfloat16, true> {
  uint4 r;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    r = *reinterpret_cast<const uint4*>(p);
  }
  __device__ __forceinline__ float at(int i) const {
    const uint32_t w = i < 2 ? r.x : i < 4 ? r.y : i < 6 ? r.z : r.w;
    return __uint_as_float(i & 1 ? w & 0xFFFF0000u : w << 16);
  }
};
template <> struct EncLoad<float, true> {
  float4 r[2];
  __device__ __forceinline__ void load(const float* p) {
    r[0] = reinterpret_cast<const float4*>(p)[0];
    r[1] = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ float at(int i) const {
    const float4& v = r[i >> 2];
    return (i & 3) == 0 ? v.x : (i & 3) == 1 ? v.y : (i & 3) == 2 ? v.z : v.w;
  }
};
// rows of any alignment, an element at a time
template <typename T> struct EncLoad<T, false> {
  float r[8];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = static_cast<float>(p[i]);
  }
  __device__ __forceinline__ float at(int i) const { return r[i]; }
};

__device__ __forceinline__ void enc_store(__nv_bfloat16* p, const float* y) {
  uint4 o;
  uint32_t* w = reinterpret_cast<uint32_t*>(&o);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = o;
}
__device__ __forceinline__ void enc_store(float* p, const float* y) {
  reinterpret_cast<float4*>(p)[0] = make_float4(y[0], y[1], y[2], y[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(y[4], y[5], y[6], y[7]);
}

// Depth of node `row`, by steps to the root (all lanes, same row).
__device__ __forceinline__ int enc_depth(const EncodeParams& p, int row, int lane) {
  int par[3];
  bool bad = false;
#pragma unroll
  for (int s = 0; s < 3; ++s) {
    const int i = lane + 32 * s;
    par[s] = 0;
    if (i >= 1 && i < p.n_rows) {
      const int v = p.parent[i];
      if (v < 0 || v >= i) bad = true;
      else par[s] = v;
    }
  }
  if (__any_sync(0xFFFFFFFFu, bad) && lane == 0) report(p.status, DFV_DEV_BAD_TREE);
  int depth = 0;
  for (int cur = row; cur > 0; ++depth) {   // par[i] < i: ends
    const int a = __shfl_sync(0xFFFFFFFFu, par[0], cur & 31);
    const int b = __shfl_sync(0xFFFFFFFFu, par[1], cur & 31);
    const int c = __shfl_sync(0xFFFFFFFFu, par[2], cur & 31);
    cur = cur < 32 ? a : cur < 64 ? b : c;
  }
  return depth;
}

template <typename TS, typename TD, int D, bool kVec>
__global__ void __launch_bounds__(kEncWarps * 32, 16)
    encode_kernel(const __grid_constant__ EncodeParams p, int near) {
  constexpr int kLanes = D / 16;         // lanes of a head
  constexpr int kHeads = 32 / kLanes;    // heads of a warp at a time
  constexpr int kAhead = sizeof(TS) == 2 ? 2 : 1;   // iterations worked on together
  const int lane = threadIdx.x & 31;
  const uint32_t task = blockIdx.x * kEncWarps + (threadIdx.x >> 5);   // below 2^27
  const int row = static_cast<int>(task / static_cast<uint32_t>(p.splits));
  grid_dep_wait();
  grid_dep_launch_dependents();   // (after the wait: see common.cuh)
  if (row >= p.n_rows) return;
  const int64_t row64 = row;
  const int j = lane % kLanes, mine = lane / kLanes;
  const int rl = p.rot >> 4;             // lanes with rotated pairs
  const bool turned = j < rl;
  const int ca = turned && !near ? 8 * j : 16 * j;
  const int cb = turned && !near ? 8 * (j + rl) : 16 * j + 8;
  // This warp's iterations [it0, it1) of the row's: the query heads', the key
  // heads', the value heads'.
  const int it0 = (static_cast<int>(task) - row * p.splits) * p.per_split;
  const int it1 = min(p.iters, it0 + p.per_split);

  // A row that is one warp's is asked for at once: its loads, an iteration or two
  // ahead, then find it on its way (78 us for 80 without).
  if (p.splits == 1) {
    constexpr int kLines = D * static_cast<int>(sizeof(TS)) / 128;   // of a head
    auto ask = [&](const void* src, int64_t stride_row, int64_t stride_head, int heads) {
      for (int i = lane; i < heads * kLines; i += 32)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(
            static_cast<const TS*>(src) + row * stride_row + (i / kLines) * stride_head +
            (i % kLines) * (128 / static_cast<int>(sizeof(TS)))));
    };
    if (p.q) ask(p.q, p.q_row, p.q_head, p.hq);
    if (p.k) ask(p.k, p.k_row, p.k_head, p.hkv);
    if (p.v) ask(p.v, p.v_row, p.v_head, p.hkv);
  }

  float cs[8], sn[8];
  if (it0 < p.it_v) {
    int64_t pos;
    if (p.positions) {
      pos = p.positions[row];
    } else {
      pos = static_cast<int64_t>(*p.ctx_len) + (p.dropped ? *p.dropped : 0);
      pos += p.parent ? enc_depth(p, row, lane) : row;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      cs[e] = 1.0f;
      sn[e] = 0.0f;
      if (turned) {
        const uint64_t t = static_cast<uint64_t>(pos) * p.turns[8 * j + e];
        // the upper half as a signed fraction of a turn, in units of half a turn
        sincospif(static_cast<float>(static_cast<int32_t>(t >> 32)) * 0x1p-31f, &sn[e], &cs[e]);
      }
    }
  }
  const bool norm = p.eps >= 0.0f;

  // Iterations [a, b) over `heads` heads at src, to dst. Loads of the next
  // iterations are in flight while one is worked on; lanes without a head work on
  // the last one and store nothing.
  EncLoad<TS, kVec> xa[2][kAhead], xb[2][kAhead];
  auto heads_of = [&](const void* src0, int64_t stride_head, void* dst0, int heads, int a, int b,
                      auto work) {
    if (a >= b) return;
    const TS* src = static_cast<const TS*>(src0);
    TD* dst = static_cast<TD*>(dst0) + row64 * heads * D;
    auto fetch = [&](int it, int s) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (it + u >= b) break;
        const TS* x = src + min((it + u) * kHeads + mine, heads - 1) * stride_head;
        xa[s][u].load(x + ca);
        xb[s][u].load(x + cb);
      }
    };
    auto turn = [&](int it, int s) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (it + u >= b) break;
        float va[8], vb[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          va[e] = xa[s][u].at(e);
          vb[e] = xb[s][u].at(e);
        }
        work(va, vb);
        const int h = (it + u) * kHeads + mine;
        if (h < heads) {
          enc_store(dst + h * D + ca, va);
          enc_store(dst + h * D + cb, vb);
        }
      }
    };
    fetch(a, 0);
    for (int it = a; it < b; it += 2 * kAhead) {
      fetch(it + kAhead, 1);
      turn(it, 0);
      fetch(it + 2 * kAhead, 0);
      turn(it + kAhead, 1);
    }
  };

  // Norm and rotation of a head: the weights are folded into the pairs' sines and
  // cosines, once for all heads; a = (a pa - b qa) r, b = (b pb + a qb) r, with
  // each element's partner as b (or a) where neighbours are pairs.
  auto turned_heads = [&](const void* src, int64_t stride_head, void* dst, int heads,
                          const float* w, int a, int b) {
    if (a >= b) return;
    float pa[8], qa[8], pb[8], qb[8];
    {
      float wa[8], wb[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) wa[e] = wb[e] = 1.0f;
      if (w) {
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
          const float4 f = *reinterpret_cast<const float4*>(w + ca + e);
          const float4 g = *reinterpret_cast<const float4*>(w + cb + e);
          wa[e] = f.x, wa[e + 1] = f.y, wa[e + 2] = f.z, wa[e + 3] = f.w;
          wb[e] = g.x, wb[e + 1] = g.y, wb[e + 2] = g.z, wb[e + 3] = g.w;
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (near) {
          pa[e] = wa[e] * cs[e >> 1];
          pb[e] = wb[e] * cs[4 + (e >> 1)];
          qa[e] = wa[e ^ 1] * ((e & 1) ? sn[e >> 1] : -sn[e >> 1]);
          qb[e] = wb[e ^ 1] * ((e & 1) ? sn[4 + (e >> 1)] : -sn[4 + (e >> 1)]);
        } else {
          pa[e] = wa[e] * cs[e];
          pb[e] = wb[e] * cs[e];
          qa[e] = -wb[e] * sn[e];
          qb[e] = wa[e] * sn[e];
        }
      }
    }
    heads_of(src, stride_head, dst, heads, a, b, [&](float* x, float* y) {
      float r = 1.0f;
      if (norm) {
        float ss = 0.0f, eps = p.eps;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(y[e], y[e], fmaf(x[e], x[e], ss));
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
        // Squares that leave float32, or vanish in it where eps does not hide
        // them: the head is brought to [1, 2) by a power of two first, and eps
        // with it (where that leaves float32, eps is all there is).
        const bool wide = ss > 1e37f || (ss < 1e-25f && eps < 1e-15f);
        if (__any_sync(0xFFFFFFFFu, wide)) {
          float m = 0.0f;
#pragma unroll
          for (int e = 0; e < 8; ++e) m = fmaxf(m, fmaxf(fabsf(x[e]), fabsf(y[e])));
#pragma unroll
          for (int o = kLanes / 2; o > 0; o >>= 1)
            m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
          const int e2 = static_cast<int>(__float_as_uint(m) >> 23);
          float sc = wide && m > 0.0f && m < INFINITY ? pow2i(max(127 - e2, -126)) : 1.0f;
          if (!(eps * sc * sc < INFINITY)) sc = 1.0f;
          eps = eps * sc * sc;
          ss = 0.0f;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            x[e] *= sc;
            y[e] *= sc;
            ss = fmaf(y[e], y[e], fmaf(x[e], x[e], ss));
          }
#pragma unroll
          for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
        }
        r = 1.0f / sqrtf(ss * (1.0f / D) + eps);
      }
      float u[8], v[8];
      if (turned && near) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          u[e] = fmaf(x[e ^ 1], qa[e], x[e] * pa[e]) * r;
          v[e] = fmaf(y[e ^ 1], qb[e], y[e] * pb[e]) * r;
        }
      } else if (turned) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          u[e] = fmaf(y[e], qa[e], x[e] * pa[e]) * r;
          v[e] = fmaf(x[e], qb[e], y[e] * pb[e]) * r;
        }
      } else {   // (no 0 * inf from a neighbour)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          u[e] = x[e] * pa[e] * r;
          v[e] = y[e] * pb[e] * r;
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] = u[e];
        y[e] = v[e];
      }
    });
  };
  if (p.q)
    turned_heads(static_cast<const TS*>(p.q) + row * p.q_row, p.q_head, p.q_out, p.hq, p.q_weight,
                 it0, min(it1, p.it_k));
  if (p.k)
    turned_heads(static_cast<const TS*>(p.k) + row * p.k_row, p.k_head, p.k_out, p.hkv,
                 p.k_weight, max(it0, p.it_k) - p.it_k, min(it1, p.it_v) - p.it_k);
  if (p.v)
    heads_of(static_cast<const TS*>(p.v) + row * p.v_row, p.v_head, p.v_out, p.hkv,
             max(it0, p.it_v) - p.it_v, it1 - p.it_v, [](float*, float*) {});
}

template <typename TS, typename TD, int D>
dfv_status encode_launch(EncodeParams p, bool near, cudaStream_t stream) {
  constexpr int kHeads = 32 / (D / 16);
  p.it_k = (p.hq + kHeads - 1) / kHeads;
  p.it_v = p.it_k + (p.hkv + kHeads - 1) / kHeads;
  p.iters = p.v ? p.it_v + (p.hkv + kHeads - 1) / kHeads : p.it_v;
  // One warp a row where that fills the GPU (the sines are computed once for
  // all of its heads); else rows are split until there are about 32 warps an SM.
  const int64_t want = (static_cast<int64_t>(sm_count()) * 32 + p.n_rows - 1) / p.n_rows;
  const int splits = static_cast<int>(want < p.iters ? want : p.iters);
  p.per_split = (p.iters + splits - 1) / splits;
  p.splits = (p.iters + p.per_split - 1) / p.per_split;
  // 16-byte loads where every row starts on such a boundary
  constexpr int64_t kE = 16 / sizeof(TS);
  auto fits = [&](const void* x, int64_t sr, int64_t sh) {
    return !x || (aligned(x, 16) && sr % kE == 0 && sh % kE == 0);
  };
  const bool vec = fits(p.q, p.q_row, p.q_head) && fits(p.k, p.k_row, p.k_head) &&
                   fits(p.v, p.v_row, p.v_head);
  cudaLaunchConfig_t cfg = {};
  const int64_t tasks = static_cast<int64_t>(p.n_rows) * p.splits;
  cfg.gridDim = dim3(static_cast<unsigned>((tasks + kEncWarps - 1) / kEncWarps));
  cfg.blockDim = dim3(kEncWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e =
      vec ? cudaLaunchKernelEx(&cfg, encode_kernel<TS, TD, D, true>, p, near ? 1 : 0)
          : cudaLaunchKernelEx(&cfg, encode_kernel<TS, TD, D, false>, p, near ? 1 : 0);
  return e == cudaSuccess ? DFV_OK : DFV_ERR_CUDA;
}

template <typename TS, typename TD>
dfv_status encode_launch_d(const EncodeParams& p, int D, bool near, cudaStream_t stream) {
  return D == 64    ? encode_launch<TS, TD, 64>(p, near, stream)
         : D == 128 ? encode_launch<TS, TD, 128>(p, near, stream)
                    : encode_launch<TS, TD, 256>(p, near, stream);
}

}  // namespace dfv

extern "C" dfv_status dfv_qk_norm_rope(
    int n_rows, int n_q_heads, int n_kv_heads, int head_dim, const void* q, const void* k,
    const void* v, int src_dtype, int64_t q_stride_row, int64_t q_stride_head,
    int64_t k_stride_row, int64_t k_stride_head, int64_t v_stride_row, int64_t v_stride_head,
    const float* q_weight, const float* k_weight, float eps, const uint64_t* turns, int rot_dim,
    int interleaved, const int32_t* positions, const int32_t* parent, const int32_t* ctx_len,
    const int32_t* dropped, void* q_out, void* k_out, void* v_out, int dst_dtype,
    uint32_t* status, dfv_stream_t stream) {
  using namespace dfv;
  if ((head_dim != 64 && head_dim != 128 && head_dim != 256) ||
      (src_dtype != DFV_DTYPE_F32 && src_dtype != DFV_DTYPE_BF16) ||
      (dst_dtype != DFV_DTYPE_F32 && dst_dtype != DFV_DTYPE_BF16))
    return DFV_ERR_UNSUPPORTED;
  if (n_rows < 0 || n_rows > (1 << 26) || n_q_heads < 0 || n_kv_heads < 0 || n_q_heads > 1024 ||
      n_kv_heads > 1024 || n_q_heads + n_kv_heads == 0 || rot_dim < 0 || rot_dim > head_dim ||
      rot_dim % 16 != 0 || eps != eps || (parent && n_rows > kMaxNodes))
    return DFV_ERR_INVALID;
  if (n_rows == 0) return DFV_OK;
  const size_t size = src_dtype == DFV_DTYPE_F32 ? 4 : 2;
  if ((n_q_heads > 0 && (!q || !q_out)) || (n_kv_heads > 0 && (!k || !k_out)) ||
      (v && (!v_out || n_kv_heads == 0)) || (rot_dim > 0 && !turns) ||
      (!positions && !ctx_len) || (positions && (parent || ctx_len || dropped)) ||
      (eps < 0.0f && (q_weight || k_weight)))
    return DFV_ERR_INVALID;
  if (!aligned(q, size) || !aligned(k, size) || !aligned(v, size) || !aligned(q_out, 16) ||
      !aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(q_weight, 16) ||
      !aligned(k_weight, 16) || !aligned(turns, 8) || !aligned(positions, 4) ||
      !aligned(parent, 4) || !aligned(ctx_len, 4) || !aligned(dropped, 4))
    return DFV_ERR_INVALID;
  const EncodeParams p = {n_rows, n_q_heads, n_kv_heads, rot_dim, 0, 0, 0, 0, 0,
                          n_q_heads > 0 ? q : nullptr, n_kv_heads > 0 ? k : nullptr, v,
                          q_stride_row, q_stride_head, k_stride_row, k_stride_head, v_stride_row,
                          v_stride_head, q_weight, k_weight, eps, turns, positions, parent,
                          ctx_len, dropped, q_out, k_out, v_out, status};
  const bool near = interleaved != 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (src_dtype == DFV_DTYPE_F32)
    return dst_dtype == DFV_DTYPE_F32 ? encode_launch_d<float, float>(p, head_dim, near, s)
                                      : encode_launch_d<float, __nv_bfloat16>(p, head_dim, near, s);
  return dst_dtype == DFV_DTYPE_F32
             ? encode_launch_d<__nv_bfloat16, float>(p, head_dim, near, s)
             : encode_launch_d<__nv_bfloat16, __nv_bfloat16>(p, head_dim, near, s);
}
