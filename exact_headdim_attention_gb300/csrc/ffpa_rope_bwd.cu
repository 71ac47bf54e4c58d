// Backward of the head norm with rotation.  With g the gradient of a row's
// output, g' = g rotated by the opposite angle (times rope_scale), xn = x r,
// r = rsqrt(mean(x^2) + eps):
//
//   dw += g' xn (over all rows),   dx = r (w g' - xn mean(w g' xn)),
//
// or dx = g' where there is no weight.  x is read again and r recomputed (a
// row sum in registers) instead of being stored by the forward.  Each row is
// read twice (x, g) and written once: the memory's bandwidth is the bound.
//
// Rows and gradients come through shared memory as in the forward, DEPTH - 1
// rows ahead (loads into registers, two rows at a time: 2.9 TB/s).
//
// dw is summed in fp32 in a fixed order (no atomics): each lane keeps its
// columns' sums over its rows in registers, a block adds its lanes and writes
// one row of partial sums, a second launch adds the blocks.
#include "ffpa_rope.cuh"

namespace ffpa {
namespace {

constexpr int RB_THREADS = 256;
constexpr int RB_BLOCKS_MAX = 512;   // blocks of queries and keys together

// Rows of the ring: more than three slow the one block of D > 512 down (T4096
// D1024: 115 us, with four 119); elsewhere four are as good or better to 2 % (T8192 D512 92, 92).
__host__ __device__ constexpr int rb_depth(int iter) { return iter == 1 ? 4 : 3; }

template <int VEC, int ITER>
__host__ __device__ constexpr int rb_row_bytes() {     // of one row and its gradient, for all threads of a block
  return RB_THREADS * ITER * 4 * VEC * 2;
}

template <bool F16, int VEC, int LPR, int ITER, bool INTER>
__global__ void __launch_bounds__(RB_THREADS, ITER == 1 ? 2 : 1) rope_bwd_kernel(const __grid_constant__ RopeParams P) {
  constexpr int GROUPS = RB_THREADS / LPR, COLS = LPR * 2 * VEC * ITER;
  constexpr int ROW = rb_row_bytes<VEC, ITER>(), PIECE = RB_THREADS * VEC * 2, RB_DEPTH = rb_depth(ITER);
  static_assert(RB_DEPTH * ROW >= GROUPS * COLS * 4, "the ring holds a block's sums");
  extern __shared__ __align__(16) char ring[];     // [RB_DEPTH][ITER][g, g, x, x][thread] vectors
  __shared__ long long freq_s[512];
  load_freqs<VEC, INTER>(P, freq_s);
  const int np = P.rot / (2 * VEC);                // rotated chunks
  const int lane = threadIdx.x % LPR, row = threadIdx.x / LPR, sub = threadIdx.x % 32 / LPR;
  const int wt = blockIdx.x < P.blocks[0] ? 0 : 1;
  const int block = blockIdx.x - (wt ? P.blocks[0] : 0);
  const RopeTensor& t = P.t[wt];
  const float inv_d = 1.0f / P.D;
  RopeChunk<VEC> ch[ITER];
  float2 w[ITER][VEC], dw[ITER][VEC];
#pragma unroll
  for (int k = 0; k < ITER; ++k) {
    ch[k] = rope_chunk<VEC>(lane + k * LPR, P.D, P.rot);
#pragma unroll
    for (int i = 0; i < VEC; ++i) dw[k][i] = make_float2(0.0f, 0.0f);
    if (ch[k].live && t.w) {
      load_weight<F16, VEC>(t.w, P.w32, ch[k].a, w[k]);
      load_weight<F16, VEC>(t.w, P.w32, ch[k].b, w[k] + VEC / 2);
    }
  }
  const unsigned stride = P.blocks[wt] * GROUPS, all = P.items[wt];
  const int per = P.heads_per[wt];
  // First head, token and number of heads of an item.
  struct Item {
    int h0, heads, b, n;
  };
  auto item_of = [&](unsigned item) {
    Item r;
    const bool in = item < all;
    const unsigned token = in ? item / P.chunks[wt] : 0;
    r.h0 = in ? (item - token * P.chunks[wt]) * per : 0;
    r.heads = in ? min(t.H - r.h0, per) : 0;
    r.b = P.B == 1 ? 0 : token / P.N;
    r.n = token - r.b * P.N;
    return r;
  };
  // Whole warps stay in the loop: the lanes of a row talk through shuffles.
  unsigned first = block * GROUPS + threadIdx.x / 32 * (32 / LPR);
  char* own = ring + threadIdx.x * (VEC * 2);
  const uint32_t own_at = smem_u32(own);
  unsigned ahead = first;
  int ahead_h = 0, ahead_heads = 0, ahead_slot = 0;
  const char *ahead_g = nullptr, *ahead_x = nullptr;
  auto issue = [&] {
    if (ahead < all) {
      if (ahead_h == 0) {
        const Item it = item_of(ahead + sub);
        ahead_heads = it.heads;
        ahead_g = P.g[wt] + it.b * P.gs[wt][0] + it.h0 * P.gs[wt][1] + it.n * P.gs[wt][2];
        ahead_x = t.x + it.b * t.xs[0] + it.h0 * t.xs[1] + it.n * t.xs[2];
      }
      if (ahead_h < ahead_heads) {
#pragma unroll
        for (int k = 0; k < ITER; ++k)
          if (ch[k].live) {
            const uint32_t to = own_at + ahead_slot * ROW + 4 * k * PIECE;
            copy_async<VEC * 2>(to, ahead_g + ch[k].a * 2);
            copy_async<VEC * 2>(to + PIECE, ahead_g + ch[k].b * 2);
            if (t.w) {
              copy_async<VEC * 2>(to + 2 * PIECE, ahead_x + ch[k].a * 2);
              copy_async<VEC * 2>(to + 3 * PIECE, ahead_x + ch[k].b * 2);
            }
          }
        ahead_g += P.gs[wt][1];
        ahead_x += t.xs[1];
      }
      if (++ahead_h == per) {
        ahead_h = 0;
        ahead += stride;
      }
      if (++ahead_slot == RB_DEPTH) ahead_slot = 0;
    }
    copy_commit();
  };
#pragma unroll 1
  for (int i = 0; i < RB_DEPTH - 1; ++i) issue();

  int ring_slot = 0;
  for (; first < all; first += stride) {
    const Item it = item_of(first + sub);
    const long long pos = P.rot ? position_of(P, it.b, it.n) : 0;
    char* to = t.y + it.b * t.ys[0] + it.h0 * t.ys[1] + it.n * t.ys[2];
    float cs[ITER][VEC], sn[ITER][VEC];
#pragma unroll
    for (int k = 0; k < ITER; ++k) {
      if (!ch[k].live || !ch[k].pair) continue;
#pragma unroll
      for (int i = 0; i < VEC; ++i) turn(pos, freq_s[i * np + lane + k * LPR], P.rope_scale, cs[k][i], sn[k][i]);
    }
#pragma unroll 1
    for (int h = 0; h < per; ++h) {
      copy_wait<RB_DEPTH - 2>();
      const char* from = own + ring_slot * ROW;
      if (++ring_slot == RB_DEPTH) ring_slot = 0;
      const bool on = h < it.heads;
      float2 g[ITER][VEC], x[ITER][VEC];
      float sq = 0.0f, dot = 0.0f;
      if (on) {
#pragma unroll
        for (int k = 0; k < ITER; ++k) {
          if (!ch[k].live) continue;
          widen<F16, VEC>(own_load<VEC>(from + 4 * k * PIECE), g[k]);
          widen<F16, VEC>(own_load<VEC>(from + (4 * k + 1) * PIECE), g[k] + VEC / 2);
          if (ch[k].pair) {
            float2 y[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
              const int p0 = pair_of<VEC, INTER>(i, 0), p1 = pair_of<VEC, INTER>(i, 1);
              const float2 z = partner<VEC, INTER>(g[k], i);
              y[i].x = g[k][i].x * cs[k][p0] + (second_of<VEC, INTER>(i, 0) ? -z.x : z.x) * sn[k][p0];
              y[i].y = g[k][i].y * cs[k][p1] + (second_of<VEC, INTER>(i, 1) ? -z.y : z.y) * sn[k][p1];
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) g[k][i] = y[i];
          }
          if (t.w) {
            widen<F16, VEC>(own_load<VEC>(from + (4 * k + 2) * PIECE), x[k]);
            widen<F16, VEC>(own_load<VEC>(from + (4 * k + 3) * PIECE), x[k] + VEC / 2);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
              sq += x[k][i].x * x[k][i].x;
              sq += x[k][i].y * x[k][i].y;
              dot += w[k][i].x * g[k][i].x * x[k][i].x;
              dot += w[k][i].y * g[k][i].y * x[k][i].y;
            }
          }
        }
      }
      issue();
      if (t.w) {
        sq = row_sum<LPR>(sq);
        dot = row_sum<LPR>(dot);
      }
      if (!on) continue;
      const float r = rsqrtf(sq * inv_d + P.eps);
      const float back = -r * dot * inv_d * r * r; // dx = (r g') w + back x
#pragma unroll
      for (int k = 0; k < ITER; ++k) {
        if (!ch[k].live) continue;
        if (t.w) {
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            g[k][i].x *= r;
            g[k][i].y *= r;
            dw[k][i].x += g[k][i].x * x[k][i].x;
            dw[k][i].y += g[k][i].y * x[k][i].y;
            g[k][i].x = g[k][i].x * w[k][i].x + back * x[k][i].x;
            g[k][i].y = g[k][i].y * w[k][i].y + back * x[k][i].y;
          }
        }
        *reinterpret_cast<Raw<VEC>*>(to + ch[k].a * 2) = narrow<F16, VEC>(g[k]);
        *reinterpret_cast<Raw<VEC>*>(to + ch[k].b * 2) = narrow<F16, VEC>(g[k] + VEC / 2);
      }
      to += t.ys[1];
    }
  }
  copy_wait<0>();
  dependents_launch();
  if (!t.w) return;
  // The block's sums, where the ring was.
  __syncthreads();
  float(*sums)[COLS] = reinterpret_cast<float(*)[COLS]>(ring);
#pragma unroll
  for (int k = 0; k < ITER; ++k) {
    if (!ch[k].live) continue;
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
      *reinterpret_cast<float2*>(&sums[row][ch[k].a + 2 * i]) = dw[k][i];
      *reinterpret_cast<float2*>(&sums[row][ch[k].b + 2 * i]) = dw[k][VEC / 2 + i];
    }
  }
  __syncthreads();
  for (int d = threadIdx.x; d < P.D; d += RB_THREADS) {
    float s = 0.0f;
    for (int i = 0; i < GROUPS; ++i) s += sums[i][d];
    P.part[wt][(int64_t)block * P.D + d] = s;
  }
}

// dw[wt][d] = sum of the blocks' partial rows: 32 columns a block, 32 threads a column.
template <bool F16>
__global__ void __launch_bounds__(1024) weight_sum_kernel(const RopeParams P) {
  const int wt = blockIdx.y;
  if (!P.dw[wt]) return;
  dependency_wait();
  const int col = threadIdx.x % 32, row = threadIdx.x / 32, d = blockIdx.x * 32 + col;
  __shared__ float sums[32][33];
  float s = 0.0f;
  if (d < P.D)
#pragma unroll 8
    for (int i = row; i < P.blocks[wt]; i += 32) s += P.part[wt][(int64_t)i * P.D + d];
  sums[row][col] = s;
  __syncthreads();
  // A warp now takes one column's 32 sums.
  s = sums[col][row];
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) s += __shfl_xor_sync(~0u, s, k);
  const int out = blockIdx.x * 32 + row;
  if (col == 0 && out < P.D) {
    if (P.w32)
      static_cast<float*>(P.dw[wt])[out] = s;
    else
      store16<F16>(static_cast<char*>(P.dw[wt]) + out * 2, s);
  }
}

template <bool F16, int VEC, int LPR, int ITER>
ffpa_status launch_bwd_as(RopeParams& P, bool inter, int sms, int dev, cudaStream_t stream) {
  const int64_t groups = RB_THREADS / LPR;
  // As many blocks as are resident, in proportion to the rows.
  const int64_t rows[2] = {(int64_t)P.items[0] * P.heads_per[0], (int64_t)P.items[1] * P.heads_per[1]};
  int64_t most = (int64_t)sms * (ITER == 1 ? 2 : 1);
  if (most > RB_BLOCKS_MAX) most = RB_BLOCKS_MAX;
  int64_t share = (most * rows[0] + (rows[0] + rows[1]) / 2) / (rows[0] + rows[1]);
  share = share < 1 ? 1 : share > most - 1 ? most - 1 : share;
  for (int i = 0; i < 2; ++i) {
    const int64_t n = (P.items[i] + groups - 1) / groups, cap = i == 0 ? share : most - share;
    P.blocks[i] = (int)(n < cap ? n : cap);
  }
  P.part[1] = P.part[0] + (int64_t)P.blocks[0] * P.D;
  const int grid = P.blocks[0] + P.blocks[1];
  const int smem = rb_depth(ITER) * rb_row_bytes<VEC, ITER>();
  auto fn = inter ? &rope_bwd_kernel<F16, VEC, LPR, ITER, true> : &rope_bwd_kernel<F16, VEC, LPR, ITER, false>;
  const ffpa_status st = set_smem_attr_once(reinterpret_cast<const void*>(fn), dev, smem);
  if (st != FFPA_OK) return st;
  fn<<<grid, RB_THREADS, smem, stream>>>(P);
  if (cudaGetLastError() != cudaSuccess) return FFPA_ERR_CUDA;
  if (P.dw[0] || P.dw[1]) {
    // A dependent launch: its blocks are set up while the first kernel runs out.
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((P.D + 31) / 32, 2);
    cfg.blockDim = dim3(1024);
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, weight_sum_kernel<F16>, P) != cudaSuccess) {
      cudaGetLastError();
      return FFPA_ERR_CUDA;
    }
  }
  return FFPA_OK;
}

template <bool F16>
ffpa_status launch_bwd_rope(RopeParams& P, bool inter, int sms, int dev, cudaStream_t stream) {
  const int64_t tokens = (int64_t)P.B * P.N;
  for (int i = 0; i < 2; ++i) {
    const int per = rope_heads(P.D, P.rot, tokens, P.t[i].H, sms);
    P.chunks[i] = (P.t[i].H + per - 1) / per;
    P.heads_per[i] = (P.t[i].H + P.chunks[i] - 1) / P.chunks[i];
    P.items[i] = (unsigned)(tokens * P.chunks[i]);
  }
  if (rope_vec(P.D, P.rot) == 8) {
    const int n = P.D / 16;
    if (n <= 4) return launch_bwd_as<F16, 8, 4, 1>(P, inter, sms, dev, stream);
    if (n <= 8) return launch_bwd_as<F16, 8, 8, 1>(P, inter, sms, dev, stream);
    if (n <= 16) return launch_bwd_as<F16, 8, 16, 1>(P, inter, sms, dev, stream);
    if (n <= 32) return launch_bwd_as<F16, 8, 32, 1>(P, inter, sms, dev, stream);
    return launch_bwd_as<F16, 8, 32, 2>(P, inter, sms, dev, stream);
  }
  const int n = P.D / 8;
  if (n <= 16) return launch_bwd_as<F16, 4, 16, 1>(P, inter, sms, dev, stream);
  if (n <= 32) return launch_bwd_as<F16, 4, 32, 1>(P, inter, sms, dev, stream);
  if (n <= 64) return launch_bwd_as<F16, 4, 32, 2>(P, inter, sms, dev, stream);
  return launch_bwd_as<F16, 4, 32, 4>(P, inter, sms, dev, stream);
}

}  // namespace
}  // namespace ffpa

extern "C" {

size_t ffpa_qk_norm_rope_bwd_workspace_bytes(int D) {
  return D < 64 || D > 1024 || D % 8 != 0 ? 0 : (size_t)ffpa::RB_BLOCKS_MAX * D * 4;
}

ffpa_status ffpa_qk_norm_rope_bwd(const void* dq_out, const void* dk_out, const void* q, const void* k, void* dq,
                                  void* dk, void* dq_weight, void* dk_weight, ffpa_dtype dt, int B, int Hq, int Hkv,
                                  int N, int D, const int64_t dqo_str[4], const int64_t dko_str[4],
                                  const int64_t q_str[4], const int64_t k_str[4], const int64_t dq_str[4],
                                  const int64_t dk_str[4], const ffpa_rope* rope, void* workspace,
                                  size_t workspace_bytes, ffpa_stream_t stream) {
  using namespace ffpa;
  RopeParams P{};
  ffpa_status st = rope_params(rope, dt, B, Hq, Hkv, N, D, &P);
  if (st != FFPA_OK) return st;
  const void* w[2] = {rope->q_weight, rope->k_weight};
  void* dw[2] = {dq_weight, dk_weight};
  const bool sums = w[0] || w[1];
  for (int i = 0; i < 2; ++i)
    if ((w[i] != nullptr) != (dw[i] != nullptr) || !on_boundary(dw[i], rope->weight_f32 ? 4 : 2)) return FFPA_ERR_INVALID;
  const bool rows = B > 0 && N > 0;
  if (!rows && !sums) return FFPA_OK;
  if (rows && (!dq_out || !dk_out || !q || !k || !dq || !dk || !dqo_str || !dko_str || !q_str || !k_str || !dq_str ||
               !dk_str))
    return FFPA_ERR_INVALID;
  if (rows && (!rows_ok(dqo_str, {B, Hq, N, D}) || !rows_ok(q_str, {B, Hq, N, D}) || !rows_ok(dq_str, {B, Hq, N, D}) ||
               !rows_ok(dko_str, {B, Hkv, N, D}) || !rows_ok(k_str, {B, Hkv, N, D}) ||
               !rows_ok(dk_str, {B, Hkv, N, D})))
    return FFPA_ERR_INVALID;
  if (rows && (!on_boundary(dq_out, 16) || !on_boundary(dk_out, 16) || !on_boundary(q, 16) || !on_boundary(k, 16) ||
               !on_boundary(dq, 16) || !on_boundary(dk, 16)))
    return FFPA_ERR_INVALID;
  if (sums && rows &&
      (!workspace || !on_boundary(workspace, 16) || workspace_bytes < ffpa_qk_norm_rope_bwd_workspace_bytes(D)))
    return FFPA_ERR_INVALID;
  int dev = 0;
  const bool turns = rows && rope->rot_dim > 0;
  auto part = [&](const void* p) { return rows ? p : nullptr; };
  st = call_device({part(dq_out), part(dk_out), part(q), part(k), part(dq), part(dk), dw[0], dw[1], w[0], w[1],
                    turns ? rope->positions : nullptr, turns ? rope->inv_freq : nullptr,
                    rows && sums ? workspace : nullptr},
                   &dev);
  if (st != FFPA_OK) return st;
  DeviceScope scope(dev);
  if (!scope.ok()) return FFPA_ERR_CUDA;
  int sms = 0;
  if ((st = call_status(dev, nullptr, &P.err, &sms)) != FFPA_OK) return st;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (!rows) {
    // No row: the weights' gradients are sums over nothing.
    for (int i = 0; i < 2; ++i)
      if (dw[i] && cudaMemsetAsync(dw[i], 0, (size_t)D * (rope->weight_f32 ? 4 : 2), s) != cudaSuccess) {
        cudaGetLastError();
        return FFPA_ERR_CUDA;
      }
    return FFPA_OK;
  }
  const void* x[2] = {q, k};
  const void* g[2] = {dq_out, dk_out};
  void* y[2] = {dq, dk};
  const int64_t* xs[2] = {q_str, k_str};
  const int64_t* gs[2] = {dqo_str, dko_str};
  const int64_t* ys[2] = {dq_str, dk_str};
  for (int i = 0; i < 2; ++i) {
    P.t[i].x = static_cast<const char*>(x[i]);
    P.t[i].y = static_cast<char*>(y[i]);
    P.g[i] = static_cast<const char*>(g[i]);
    P.dw[i] = dw[i];
    for (int j = 0; j < 3; ++j) {
      P.t[i].xs[j] = xs[i][j] * 2;
      P.t[i].ys[j] = ys[i][j] * 2;
      P.gs[i][j] = gs[i][j] * 2;
    }
  }
  P.part[0] = static_cast<float*>(workspace);
  return dt == FFPA_FP16 ? launch_bwd_rope<true>(P, rope->interleaved != 0, sms, dev, s)
                         : launch_bwd_rope<false>(P, rope->interleaved != 0, sms, dev, s);
}

}  // extern "C"
