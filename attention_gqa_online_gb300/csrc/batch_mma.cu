// batch_mma.cu -- attention of each sequence's new tokens over its pages with
// warp-level tensor-core products (m16n8k16), for every layout the batched call
// takes, the kernel that joins its split items, and the choice of kernel.
//
//   s_j = scale q.k_j;  s_j = cap tanh(s_j / cap);  s_j -= slope |p - j|
//   out = sum_j softmax(s)_j v_j over the row's keys [lo, hi)
//
// One thread block (4 warps) walks its range of items (batch_plan.cuh) with
// blocks of 64 flattened rows, 16 a warp, and tiles of 64 keys: K and V rows
// come through the block table by 16-byte asynchronous copies into a
// two-stage ring (rows outside the block's windows arrive as zeros, whatever
// the pages hold there), scores and the running max and sum stay in fp32
// registers, and P is rounded to the cache's type for the second product.
//
// Only pages that are no whole 8-row groups come here: the other kernels fetch
// boxes of 8 to 128 rows (they could fetch single rows, as they do at the ends
// of windows, but have no form of it for whole tiles). Bound by its products and
// row-wise copies: 2 chunks of 512 at 8192, 32 heads over 8 of 128, bf16, in 767
// us with pages of 4 rows (tcgen05, pages of 16: 110), 64 single tokens of 8192
// in 854 (310).
#include <atomic>
#include <cfloat>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <type_traits>

#include "batch.h"
#include "batch_plan.cuh"
#include "batch_score.cuh"
#include "cache8.cuh"
#include "common.cuh"
#include "internal.h"
#include "mma16.cuh"

namespace attn {
namespace {

constexpr int kRows = 64, kKeys = 64, kThreads = 128, kStages = 2;
constexpr int kItemCost = 2;  // tiles

// A tile is rows of DP 16-bit elements; 16-byte unit u of row r sits at unit
// u ^ (r & 7), so ldmatrix reads eight rows without bank conflicts.
template <int DP>
__device__ __forceinline__ uint32_t unit_addr(uint32_t base, int r, int u) {
  return base + (uint32_t)(r * DP * 2 + 16 * (u ^ (r & 7)));
}

template <int DP>
struct MmaSmem {
  unsigned char q[kRows * DP * 2];
  unsigned char k[kStages][kKeys * DP * 2];
  unsigned char v[kStages][kKeys * DP * 2];
};

// T: of Q and the result.  C8: K and V are codes of cache8.cuh, and operands fp16.
template <typename T, int DP, bool CAP, bool SINKS, bool C8>
__global__ void __launch_bounds__(kThreads) batch_mma_kernel(const BatchArgs a, const ScoreMap sm) {
  using TO = typename std::conditional<C8, __half, T>::type;
  extern __shared__ __align__(128) unsigned char smem_raw[];
  MmaSmem<DP>& sh = *reinterpret_cast<MmaSmem<DP>*>(smem_raw);
  __shared__ plan::Start start;
  __shared__ long long warp_sums[kThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  plan::make_plan<kRows, kKeys, kThreads, SINKS>(a, blockIdx.x, gridDim.x, reinterpret_cast<int*>(smem_raw), warp_sums, &start);
  BatchSplit split{};
  plan::Walker<kRows, kKeys, SINKS> walk(a, start);
  plan::Piece p;
  const uint32_t q_base = smem_u32(sh.q);
  constexpr int kUnits = DP / 8;
  while (walk.next(p, &split)) {
    __syncthreads();  // the previous piece (or the plan) no longer reads shared memory
    const int rows = min(kRows, p.q.q_len * a.gs - p.b * kRows);
    // Q block; rows and columns past the data are zeros.
    for (int i = tid; i < kRows * kUnits; i += kThreads) {
      const int r = i / kUnits, u = i % kUnits;
      const int f = p.b * kRows + r, t = plan::token_of(a, f), h = p.g * a.gs + f - t * a.gs;
      const bool ok = r < rows && 8 * u < a.D;
      const T* src = static_cast<const T*>(a.q);
      if (ok) src += (long long)(p.q.row0 + t) * a.q_stride + (long long)h * a.D + 8 * u;
      cp_async16(sh.q + r * DP * 2 + 16 * (u ^ (r & 7)), src, ok ? 16u : 0u);
    }
    const uint32_t* table = a.block_table + (long long)p.s * a.max_blocks;
    const int tile0 = plan::first_tile<SINKS>(p.k) + p.t0;  // the piece's first tile, as plan::tile_at counts
    auto load_tile = [&](int i, int st) {
      const int key0 = plan::tile_at<SINKS>(i, p.k.ns, p.k.skip) * kKeys;
      for (int c = tid; c < kKeys * kUnits; c += kThreads) {
        const int r = c / kUnits, u = c % kUnits;
        const int key = key0 + r;
        long long row = -1;
        if ((key >= p.k.lo_min && key < p.k.hi_max) || (SINKS && key < p.k.se))
          row = paged_row(table, a.page_rows, a.num_pages, key, a.status);
        const bool ok = row >= 0 && 8 * u < a.D;
        if constexpr (C8) {
          const long long block = ok ? (long long)divide((uint32_t)row, a.by_scale) * a.G + p.g : 0;
          auto eight = [&](const void* pages, const uint8_t* scales, unsigned char* dst) {
            uint4 w = make_uint4(0u, 0u, 0u, 0u);
            if (ok) {
              const uint2 c8 = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(pages) + row * a.kv_dim +
                                                               (long long)p.g * a.D + 8 * u);
              const uint32_t mul = c8::pow2_half2(c8::exp_of(scales[block]));
              c8::to_half4(c8.x, w.x, w.y);
              c8::to_half4(c8.y, w.z, w.w);
              w = make_uint4(c8::mul_half2(w.x, mul), c8::mul_half2(w.y, mul), c8::mul_half2(w.z, mul),
                             c8::mul_half2(w.w, mul));
            }
            *reinterpret_cast<uint4*>(dst + r * DP * 2 + 16 * (u ^ (r & 7))) = w;
          };
          eight(a.k_pages, a.k_scales, sh.k[st]);
          eight(a.v_pages, a.v_scales, sh.v[st]);
          continue;
        }
        const long long off = ok ? row * a.kv_dim + (long long)p.g * a.D + 8 * u : 0;
        const int dst = r * DP * 2 + 16 * (u ^ (r & 7));
        cp_async16(sh.k[st] + dst, static_cast<const T*>(a.k_pages) + off, ok ? 16u : 0u);
        cp_async16(sh.v[st] + dst, static_cast<const T*>(a.v_pages) + off, ok ? 16u : 0u);
      }
    };
    const int n = p.t1 - p.t0;
    if (n > 0) load_tile(tile0, 0);
    cp_async_commit();

    // This thread's rows: r0 = 16 warp + lane/4 and r0 + 8.
    int lo[2], hi[2], pos[2];
    float slope[2], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = 16 * warp + (lane >> 2) + 8 * e;
      const int f = p.b * kRows + min(r, rows - 1), t = plan::token_of(a, f);
      lo[e] = plan::row_lo(a, p.q, t);
      hi[e] = r < rows ? plan::row_hi(p.q, t) : 0;
      pos[e] = p.q.len - p.q.q_len + t;
      slope[e] = a.slopes != nullptr ? a.slopes[p.g * a.gs + f - t * a.gs] * kLog2e : 0.f;
    }
    float o[DP / 8][4];
#pragma unroll
    for (int i = 0; i < DP / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;

    float qf[2] = {1.f, 1.f};  // powers of two that came off the rows of Q (rows r0 and r0 + 8)
    if constexpr (C8 && !std::is_same<T, __half>::value) {
      cp_async_wait<0>();
      __syncthreads();
      // Two lanes a row, every other unit.
      const int r = 16 * warp + (lane >> 1);
      unsigned char* row = sh.q + r * DP * 2;
      float m = 0.f;
      for (int u = lane & 1; u < kUnits; u += 2) m = fmaxf(m, q16::largest(row + 16 * (u ^ (r & 7))));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      const int E = pow2_scale_exp(m);
      for (int u = lane & 1; u < kUnits; u += 2) q16::to_half(row + 16 * (u ^ (r & 7)), pow2f(14 - E));
      const float f = pow2f(E - 14);
      qf[0] = __shfl_sync(0xffffffffu, f, 2 * (lane >> 2));
      qf[1] = __shfl_sync(0xffffffffu, f, 2 * (lane >> 2) + 16);
      __syncwarp();  // the warp's own rows: it alone reads them
    }
    for (int i = 0; i < n; ++i) {
      const int st = i % kStages;
      if (i + 1 < n) load_tile(tile0 + i + 1, (i + 1) % kStages);
      cp_async_commit();
      cp_async_wait<1>();
      __syncthreads();
      const uint32_t k_base = smem_u32(sh.k[st]), v_base = smem_u32(sh.v[st]);
      float s[kKeys / 8][4];
#pragma unroll
      for (int j = 0; j < kKeys / 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[j][e] = 0.f;
#pragma unroll
      for (int c = 0; c < DP / 16; ++c) {
        uint32_t qa[4];
        ldsm4(qa, unit_addr<DP>(q_base, 16 * warp + (lane & 15), 2 * c + (lane >> 4)));
#pragma unroll
        for (int j = 0; j < kKeys / 16; ++j) {  // 16 keys: units 2c, 2c+1 of two 8-row groups
          uint32_t kb[4];
          ldsm4(kb, unit_addr<DP>(k_base, 16 * j + (lane & 7) + 8 * (lane >> 4), 2 * c + ((lane >> 3) & 1)));
          mma16816<TO>(s[2 * j], qa, kb[0], kb[1]);
          mma16816<TO>(s[2 * j + 1], qa, kb[2], kb[3]);
        }
      }
      const int key0 = plan::tile_at<SINKS>(tile0 + i, p.k.ns, p.k.skip) * kKeys;
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int j = 0; j < kKeys / 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = key0 + 8 * j + 2 * (lane & 3) + (e & 1), x = e >> 1;
          float v = s[j][e];
          if (C8) v *= qf[x];
          if (CAP) {
            v = sm.out_mul * tanh_score(v * sm.in_mul);
          } else {
            v *= sm.scale2;
          }
          v -= slope[x] * fabsf((float)(pos[x] - key));
          v = ((key >= lo[x] || (SINKS && key < a.sinks)) && key < hi[x]) ? v : -INFINITY;
          s[j][e] = v;
          mx[x] = fmaxf(mx[x], v);
        }
      float corr[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], 1));
        mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], 2));
        const float mn = fmaxf(m[x], mx[x]);
        corr[x] = (mn == m[x]) ? 1.f : ex2(m[x] - mn);
        m[x] = mn;
        l[x] *= corr[x];
      }
      constexpr float kHead = std::is_same<TO, __half>::value ? kF16Head : 0.f;
      const float sub[2] = {m[0] == -INFINITY ? 0.f : m[0] - kHead, m[1] == -INFINITY ? 0.f : m[1] - kHead};
#pragma unroll
      for (int j = 0; j < DP / 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][e] *= corr[e >> 1];
      // P (fp32 sum, then rounded to the operand type) times V.
#pragma unroll
      for (int j = 0; j < kKeys / 16; ++j) {
        float pr[2][4];
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            pr[y][e] = ex2(s[2 * j + y][e] - sub[e >> 1]);
            l[e >> 1] += pr[y][e];
          }
        const uint32_t pa[4] = {pack2<TO>(pr[0][0], pr[0][1]), pack2<TO>(pr[0][2], pr[0][3]),
                                pack2<TO>(pr[1][0], pr[1][1]), pack2<TO>(pr[1][2], pr[1][3])};
#pragma unroll
        for (int c = 0; c < DP / 16; ++c) {
          uint32_t vb[4];
          ldsm4_t(vb, unit_addr<DP>(v_base, 16 * j + (lane & 15), 2 * c + (lane >> 4)));
          mma16816<TO>(o[2 * c], pa, vb[0], vb[1]);
          mma16816<TO>(o[2 * c + 1], pa, vb[2], vb[3]);
        }
      }
      __syncthreads();  // the stage may be refilled
    }
    cp_async_wait<0>();
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int r = 16 * warp + (lane >> 2) + 8 * x;
      if (r >= rows) continue;
      if (p.whole) {
        const float inv = l[x] == 0.f ? 0.f : 1.f / l[x];
        const int f = p.b * kRows + r, t = plan::token_of(a, f), h = p.g * a.gs + f - t * a.gs;
        T* dst = static_cast<T*>(a.out) + (long long)(p.q.row0 + t) * a.out_stride + (long long)h * a.D;
#pragma unroll
        for (int c = 0; c < DP / 8; ++c) {
          const int d = 8 * c + 2 * (lane & 3);
          if (d < a.D) *reinterpret_cast<uint32_t*>(dst + d) = pack2<T>(o[c][2 * x] * inv, o[c][2 * x + 1] * inv);
        }
      } else {
        float* part = a.partial + (long long)(2 * blockIdx.x + p.slot) * kRows * (a.D + 2);
#pragma unroll
        for (int c = 0; c < DP / 8; ++c) {
          const int d = 8 * c + 2 * (lane & 3);
          if (d < a.D) *reinterpret_cast<float2*>(part + r * a.D + d) = make_float2(o[c][2 * x], o[c][2 * x + 1]);
        }
        if ((lane & 3) == 0)
          *reinterpret_cast<float2*>(part + (long long)kRows * a.D + 2 * r) = make_float2(m[x], l[x]);
      }
    }
  }
  if (tid == 0) a.split[blockIdx.x] = split;
}

// Joins the pieces of a split item: out = sum_i 2^(m_i - m) O_i / sum_i
// 2^(m_i - m) l_i, pieces in key order.  Grid (blocks of the attention grid,
// row groups); a block without a split item leaves at once.
constexpr int kJoinThreads = 128;
template <typename T>
__global__ void __launch_bounds__(kJoinThreads) batch_combine_kernel(const BatchArgs a) {
  grid_dependency_wait();
  const BatchSplit sp = a.split[blockIdx.x];
  if (!sp.valid) return;
  const plan::SeqInfo q = plan::load_seq(a, sp.seq);
  const int rows = min(kRows, q.q_len * a.gs - sp.blk * kRows);
  const int tpr = a.D / 4;  // threads per row, four columns each
  const long long slot_floats = (long long)kRows * (a.D + 2);
  const int per = kJoinThreads / tpr;
  const int sub = threadIdx.x / tpr, col = 4 * (threadIdx.x % tpr);
  if (sub >= per) return;
  const float* first = a.partial + (2ll * blockIdx.x + sp.slot0) * slot_floats;
  for (int r = blockIdx.y * per + sub; r < rows; r += gridDim.y * per) {
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = blockIdx.x; c <= sp.last; ++c) {
      const float* part = c == (int)blockIdx.x ? first : a.partial + 2ll * c * slot_floats;
      const float2 ml = *reinterpret_cast<const float2*>(part + (long long)kRows * a.D + 2 * r);
      const float4 v = *reinterpret_cast<const float4*>(part + (long long)r * a.D + col);
      if (ml.y == 0.f) continue;  // the piece holds none of the row's keys
      const float mn = fmaxf(m, ml.x);
      const float f0 = l == 0.f ? 0.f : ex2(m - mn), f1 = ex2(ml.x - mn);
      o = make_float4(o.x * f0 + v.x * f1, o.y * f0 + v.y * f1, o.z * f0 + v.z * f1, o.w * f0 + v.w * f1);
      l = l * f0 + ml.y * f1;
      m = mn;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int f = sp.blk * kRows + r, t = plan::token_of(a, f), h = sp.g * a.gs + f - t * a.gs;
    T* dst = static_cast<T*>(a.out) + (long long)(q.row0 + t) * a.out_stride + (long long)h * a.D + col;
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<T>(o.x * inv, o.y * inv), pack2<T>(o.z * inv, o.w * inv));
  }
}

template <typename T, int DP>
int launch_mma_t(const BatchArgs& a, int blocks, cudaStream_t s) {
  const ScoreMap sm = score_map(a);
  const size_t plan_bytes = ((size_t)a.n_seqs + 1) * sizeof(int);
  const size_t smem = sizeof(MmaSmem<DP>) > plan_bytes ? sizeof(MmaSmem<DP>) : plan_bytes;
  // (Codes have one form.)
  auto of_cap = [&](auto cap) {
    constexpr bool CAP = decltype(cap)::value;
    return a.k_scales != nullptr ? batch_mma_kernel<T, DP, CAP, true, true>
           : a.sinks > 0         ? batch_mma_kernel<T, DP, CAP, true, false>
                                 : batch_mma_kernel<T, DP, CAP, false, false>;
  };
  auto kern = a.softcap > 0.f ? of_cap(std::true_type{}) : of_cap(std::false_type{});
  if (!set_smem_limit(reinterpret_cast<const void*>(kern), smem)) return ATTN_ERR_CUDA;
  BatchArgs b = a;
  b.item_cost = kItemCost;
  kern<<<blocks, kThreads, smem, s>>>(b, sm);
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

template <typename T>
int launch_combine_t(const BatchArgs& a, int blocks, cudaStream_t s) {
  BatchArgs b = a;
  void* args[] = {&b};
  return launch_pdl(reinterpret_cast<const void*>(batch_combine_kernel<T>), dim3(blocks, 4), dim3(kJoinThreads), 0, s,
                    args) == cudaSuccess
             ? ATTN_OK
             : ATTN_ERR_CUDA;
}

}  // namespace

int launch_batch_mma(const BatchArgs& a, int dtype, int blocks, cudaStream_t s) {
  if (dtype == ATTN_DT_BF16)
    return a.D <= 64 ? launch_mma_t<__nv_bfloat16, 64>(a, blocks, s) : launch_mma_t<__nv_bfloat16, 128>(a, blocks, s);
  return a.D <= 64 ? launch_mma_t<__half, 64>(a, blocks, s) : launch_mma_t<__half, 128>(a, blocks, s);
}

static int launch_batch_combine(const BatchArgs& a, int dtype, int blocks, cudaStream_t s) {
  return dtype == ATTN_DT_BF16 ? launch_combine_t<__nv_bfloat16>(a, blocks, s) : launch_combine_t<__half>(a, blocks, s);
}

// Calls begun (a line of its own), arrival counters, split records, and partial slots (two a thread block; at most 128 rows a multiprocessor).
constexpr size_t kCallsBytes = 128;
size_t batch_workspace_bytes(int head_dim, int sm_count) {
  const int D = head_dim <= 64 ? 64 : 128;  // as the kernels round it up
  return (size_t)2 * sm_count * 128 * (D + 2) * sizeof(float) + (size_t)2 * sm_count * sizeof(BatchSplit) +
         (size_t)4 * ((sm_count + 7) / 8 * 8) * sizeof(unsigned long long) + kCallsBytes;
}

static std::atomic<unsigned> g_wait_ns{0};
void set_batch_wait_ns(unsigned ns) { g_wait_ns = ns; }

int launch_batch_paged(BatchArgs a, int dtype, void* workspace, int sm_count, cudaStream_t s) {
  a.by_gs = fast_div((uint32_t)a.gs);
  a.by_page = fast_div((uint32_t)a.page_rows);
  a.by_scale = fast_div((uint32_t)a.scale_rows);
  a.wait_ns = g_wait_ns.load(std::memory_order_relaxed);
  a.calls = static_cast<unsigned long long*>(workspace);
  a.arrived = a.calls + kCallsBytes / sizeof(unsigned long long);
  a.split = reinterpret_cast<BatchSplit*>(a.arrived + 4 * ((sm_count + 7) / 8 * 8));
  a.partial = reinterpret_cast<float*>(a.split + 2 * sm_count);
  // Pages move by TMA boxes of the largest power of two of rows that divides a
  // page, whole 8-row groups of the swizzle; other pages take the mma kernel.
  int box = a.page_rows & -a.page_rows;
  if (box > 128) box = 128;
  const bool codes = a.k_scales != nullptr;
  if (box >= 8) {
    // About one row a sequence: the kernel of 16-row blocks. 64 sequences of 8192 positions, 8 kv heads of 128: 308
    // us at 4 query heads a kv head, 313 at 16 (tcgen05 kernel: 317 and 322); heads of 64: 162 (187); 8 sequences of
    // 2048: 16 us against 24. More heads a kv head would read K and V once for every 16 of them. The lengths are on the
    // device, so a call with as many sequences as rows comes here even if one sequence has them all, and its K and V
    // are read once for every 16 rows: a chunk of 250 at 4096, 38 us by itself, takes 111 among 255 idle sequences.
    // Over codes, 64 sequences of 8192: 208 us at 1 to 16 query heads a kv head (tcgen05 631); 8 of 2048 23 (48). The rule is
    // that of 16 bits, and late for codes: 16 sequences of 4096, 4 heads a kv head, with 2, 4, 8, 16, 32 tokens 44, 44, 64, 107,
    // 195 us here and 97, 98, 99, 105, 99 there (16 bits: 64, 66, 101, 158 and 72, 72, 72, 87).
    if (a.total_rows <= (uint32_t)a.n_seqs && a.gs <= 16) return launch_batch_decode(a, dtype, sm_count, box, s);
    // Pairs of multiprocessors share K and V tiles between 256 rows, where sequences have that many on average (a long
    // chunk beside many single tokens does not get them: 2048 tokens at 4096 and 63 single tokens 232 us, apart 91 and 158). 16
    // sequences of 4096, 4 heads a kv head of 128, with 32, 64, 128, 256, 512, 1024 rows a kv head: pairs 64, 74, 77,
    // 76, 120, 210 us, single blocks 57, 71, 74, 99, 164, 312. Over codes, at 128, 256, 512, 1024 rows: pairs 136, 126, 222, 406,
    // single blocks 99, 177, 324, 609.
    if (a.D > 64 && 128 % a.gs == 0 && sm_count % 2 == 0 && (long long)a.total_rows * a.gs >= 256ll * a.n_seqs)
      return codes        ? launch_batch_tc_codes_pair(a, dtype, sm_count, box, s)
             : a.sinks > 0 ? launch_batch_tc_sinks_pair(a, dtype, sm_count, box, s)
             : a.D == 128 ? launch_batch_tc_pair(a, dtype, sm_count, box, s)
                          : launch_batch_tc_part_pair(a, dtype, sm_count, box, s);
    if (a.D > 64)
      return codes         ? launch_batch_tc_codes128(a, dtype, sm_count, box, s)
             : a.sinks > 0 ? launch_batch_tc_sinks128(a, dtype, sm_count, box, s)
             : a.D == 128 ? launch_batch_tc_d128(a, dtype, sm_count, box, s)
                          : launch_batch_tc_part128(a, dtype, sm_count, box, s);
    return codes         ? launch_batch_tc_codes64(a, dtype, sm_count, box, s)
           : a.sinks > 0 ? launch_batch_tc_sinks64(a, dtype, sm_count, box, s)
           : a.D == 64 ? launch_batch_tc_d64(a, dtype, sm_count, box, s)
                       : launch_batch_tc_part64(a, dtype, sm_count, box, s);
  }
  const int rc = launch_batch_mma(a, dtype, 2 * sm_count, s);
  return rc != ATTN_OK ? rc : launch_batch_combine(a, dtype, 2 * sm_count, s);
}

}  // namespace attn
