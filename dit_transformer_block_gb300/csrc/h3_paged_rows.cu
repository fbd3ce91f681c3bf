// Attention of single rows over short paged sequences: a row and up to eight of the
// heads on a key head at a time.
//
// The products are 8 by keys by 128: bound by the bytes of the keys and values, or,
// for a few rows, by latency. So the warps take the 16-key chunks in turn, each with
// a maximum, sum and O of its own: a chunk's 8 KB are all requested at once, straight
// into the registers of a warp's own 16 x 8 x 16 products, and the scores leave one
// product where the next one takes its weights from. The warps meet once, in shared
// memory, and where rows are few a cluster of CTAs shares the keys of one. A short
// sequence is then three loads deep (the row's sequence, its page, the keys and
// values); the tensor-memory kernel (h3_paged_attention.cu), which takes everything
// else, has its setup, five kinds of warps and their hand-offs on top of that.
//
// Measured (a call, graph replay): one row, 4 heads, 250 keys 5.3 us, 4,000 keys
// 8.5 us, both latency (a CTA reads 70 GB/s, so the keys are spread over CTAs);
// 1,024 rows of 256 keys, 42 heads on 42 845 us (6.7 TB/s of 5.6 GB), 32 on 8 175 us
// (6.1 TB/s of 1.07 GB).
#include <cuda_bf16.h>

#include <algorithm>

#include "h3_internal.cuh"
#include "h3_ptx.cuh"

namespace h3 {
namespace {

constexpr int PR_DH = 128;
constexpr int PR_HEADS = 8;  // query heads of a CTA
constexpr int PR_MAX_WARPS = 8;
constexpr int PR_CHUNK = 16;  // keys of a chunk; a page has one or several

struct RowsArgs {
  PagedBatch b;
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  __nv_bfloat16* o;
  int64_t ld_q, ld_o;
  int Hkv, G;
  int groups, sets;  // of PR_HEADS heads on a key head, on all of them
  int cluster;       // CTAs per row and group of heads
  float scale_log2;  // softmax_scale * log2(e)
  int causal;
  const int32_t* prefix_pages;
  int prefix_len;
  float* part_o;   // not NULL: [T * H][128] sums and
  float* part_ml;  // [T * H] (maximum, sum) go there instead of the output
};

// D += A B of one warp: A 16 x 16, B 16 x 8, bf16 in, FP32 out.
__device__ __forceinline__ void mma_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                            uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A (row, head)'s result while its parts are joined, four channels per lane.
struct Joined {
  float m = -INFINITY, l = 0.f;  // maximum -inf: no key (see KEYS_SEEN)
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);

  __device__ __forceinline__ void add(float2 ml, const float4& y) {
    const float top = fmaxf(m, ml.x);
    if (top == -INFINITY) return;  // no key so far
    const float f = ex2_approx(m - top), w = ex2_approx(ml.x - top);
    m = top;
    l = fmaf(ml.y, w, l * f);
    o.x = fmaf(y.x, w, o.x * f);
    o.y = fmaf(y.y, w, o.y * f);
    o.z = fmaf(y.z, w, o.z * f);
    o.w = fmaf(y.w, w, o.w * f);
  }
  __device__ __forceinline__ void add(float2 ml, const float* part, int lane) {
    add(ml, reinterpret_cast<const float4*>(part)[lane]);
  }
  // of the cluster's CTA r, at these places of its shared memory
  __device__ __forceinline__ void add_peer(uint32_t ml, uint32_t part, int r, int lane) {
    float2 p;
    float4 y;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                 : "=f"(p.x), "=f"(p.y)
                 : "r"(mapa_shared(ml, r))
                 : "memory");
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(y.x), "=f"(y.y), "=f"(y.z), "=f"(y.w)
                 : "r"(mapa_shared(part, r) + lane * 16)
                 : "memory");
    add(p, y);
  }
  __device__ __forceinline__ void store(const RowsArgs& a, int t, int head, int lane) const {
    if (a.part_o != nullptr) {
      const int64_t at = static_cast<int64_t>(t) * (a.Hkv * a.G) + head;
      reinterpret_cast<float4*>(a.part_o + at * PR_DH)[lane] = o;
      if (lane == 0) *reinterpret_cast<float2*>(a.part_ml + at * 2) = make_float2(m, l);
      return;
    }
    const float inv = m == -INFINITY ? 0.f : 1.0f / l;  // no key: zeros
    *reinterpret_cast<uint2*>(a.o + t * a.ld_o + head * PR_DH + lane * 4) =
        make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
  }
};

// CTAS: per SM, that the registers have to allow (2: 128 registers and 16 bytes of
// spills, 11 % slower alone and as much faster where an SM has several).
template <int CTAS>
__global__ void __launch_bounds__(32 * PR_MAX_WARPS, CTAS)
    paged_rows_kernel(const RowsArgs a) {
  extern __shared__ float sm[];  // [warps][heads][128] O, then [warps][heads] (max, sum)
  const unsigned unit = blockIdx.x / a.cluster;
  const int rank = static_cast<int>(blockIdx.x % a.cluster);
  const int t = static_cast<int>(unit / a.sets), set = static_cast<int>(unit % a.sets);
  const int hk = set / a.groups, head0 = hk * a.G + set % a.groups * PR_HEADS;
  const int heads = min(PR_HEADS, (hk + 1) * a.G - head0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int warp0 = rank * warps + warp, step = a.cluster * warps;
  // a kernel that goes on from the partial results may take SMs that become free
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // In a product this lane has row (of A and D; also row n + 8) or column (of B) n,
  // and of the contraction the places 2 c, 2 c + 1, 2 c + 8 and 2 c + 9; of D columns
  // 2 c and 2 c + 1. Scores are q k^T (rows: heads), and which channel has which place
  // is free as long as q and k agree: the places of steps 2 i and 2 i + 1 are the
  // eight channels from 32 i + 8 c on, one 16-byte load. The output is v^T p^T (rows:
  // channels), whose B is what the scores' D holds; rows n and n + 8 of tile (i, j)
  // are channels 64 i + 8 n + 2 j and the next, so a 16-byte load holds four tiles.
  const int n = lane >> 2, c = lane & 3;

  uint32_t q[16] = {};
  if (n < heads) {
    const uint4* qrow = reinterpret_cast<const uint4*>(a.q + t * a.ld_q) + (head0 + n) * 16 + c;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 x = __ldg(qrow + i * 4);
      q[4 * i] = x.x;
      q[4 * i + 1] = x.y;
      q[4 * i + 2] = x.z;
      q[4 * i + 3] = x.w;
    }
  }

  // the row's sequence, bounded as in the tensor-core kernel
  const int b = ends_up_to(a.b.cu_q, a.b.B, t);
  if (b >= a.b.B) return;
  const int c0 = min(max(__ldg(a.b.cu_q + b), 0), a.b.T);
  const int q_len = min(max(__ldg(a.b.cu_q + b + 1), c0), a.b.T) - c0;
  if (t < c0 || t >= c0 + q_len) return;
  const int len = max(__ldg(a.b.kv_len + b), 0);
  int own = min(len, a.b.max_pages << a.b.page_log2);  // own keys that the row sees
  if (a.causal) own = min(max(len - q_len + (t - c0) + 1, 0), own);
  const int32_t* table = a.b.page_table + static_cast<int64_t>(b) * a.b.max_pages;
  const int pre = (a.prefix_len + PR_CHUNK - 1) / PR_CHUNK;  // chunks of the prefix
  const int chunks = pre + (own + PR_CHUNK - 1) / PR_CHUNK;

  float o[2][4][4] = {};  // heads 2 c, 2 c + 1 of a channel, then of the next
  float m = -INFINITY, l = 0.f;
  int page = 0;  // of the warp's chunk it + lane
#pragma unroll 1
  for (int it = 0; warp0 + it * step < chunks; ++it) {
    const int ch = warp0 + it * step;
    if ((it & 31) == 0) {
      const int mine = ch + lane * step;
      page = -1;
      if (mine < pre)
        page = __ldg(a.prefix_pages + (static_cast<int64_t>(mine) * PR_CHUNK >> a.b.page_log2));
      else if (mine < chunks)
        page = __ldg(table + (static_cast<int64_t>(mine - pre) * PR_CHUNK >> a.b.page_log2));
    }
    const int p = __shfl_sync(0xffffffffu, page, it & 31);
    const int j0 = (ch < pre ? ch : ch - pre) * PR_CHUNK;
    const int live = (ch < pre ? a.prefix_len : own) - j0;  // keys of the chunk, if below 16
    const int lim = p >= 0 && p < a.b.num_pages ? live : 0;  // those in memory, else zeros
    const int64_t row = ((static_cast<int64_t>(lim > 0 ? p : 0) * a.Hkv + hk) << a.b.page_log2) +
                        (j0 & ((1 << a.b.page_log2) - 1));
    const uint4* kp = reinterpret_cast<const uint4*>(a.k) + (row + n) * 16 + c;
    const uint4* vp = reinterpret_cast<const uint4*>(a.v) + (row + 2 * c) * 16 + n;
    uint4 kx[2][4], vx[4][2];
#pragma unroll
    for (int h = 0; h < 2; ++h)  // key 8 h + n
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        kx[h][i] = make_uint4(0, 0, 0, 0);
        if (8 * h + n < lim) kx[h][i] = __ldg(kp + h * 128 + i * 4);
      }
#pragma unroll
    for (int w = 0; w < 4; ++w)  // keys 2 c, 2 c + 1, 2 c + 8, 2 c + 9
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int key = (w >> 1) * 8 + (w & 1);
        vx[w][i] = make_uint4(0, 0, 0, 0);
        if (2 * c + key < lim) vx[w][i] = __ldg(vp + key * 16 + i * 8);
      }
    float s[2][4] = {};  // keys 8 h + 2 c, + 1 of head n (the rows from 8 on are unused)
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        mma_16x8x16(s[h], q[4 * i], 0u, q[4 * i + 1], 0u, kx[h][i].x, kx[h][i].y);
        mma_16x8x16(s[h], q[4 * i + 2], 0u, q[4 * i + 3], 0u, kx[h][i].z, kx[h][i].w);
      }
    float z[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      z[i] = (i >> 1) * 8 + 2 * c + (i & 1) < live ? s[i >> 1][i & 1] * a.scale_log2 : -INFINITY;
    float mx = fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3]));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    if (__any_sync(0xffffffffu, mx > m)) {
      const float top = fmaxf(m, mx);
      const float f = m == top ? 1.f : ex2_approx(m - top);  // 0 from -inf
      m = top;
      l *= f;
      const float f0 = __shfl_sync(0xffffffffu, f, 8 * c);      // of head 2 c
      const float f1 = __shfl_sync(0xffffffffu, f, 8 * c + 4);  // and the next
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          o[i][j][0] *= f0;
          o[i][j][1] *= f1;
          o[i][j][2] *= f0;
          o[i][j][3] *= f1;
        }
    }
    const float top = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      z[i] = ex2_approx(z[i] - top);
      l += z[i];
    }
    // rounded to bf16, the type of V in the product; the sum is of the unrounded
    const uint32_t w0 = pack_bf16x2(z[0], z[1]), w1 = pack_bf16x2(z[2], z[3]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t x[4][4] = {{vx[0][i].x, vx[0][i].y, vx[0][i].z, vx[0][i].w},
                                {vx[1][i].x, vx[1][i].y, vx[1][i].z, vx[1][i].w},
                                {vx[2][i].x, vx[2][i].y, vx[2][i].z, vx[2][i].w},
                                {vx[3][i].x, vx[3][i].y, vx[3][i].z, vx[3][i].w}};
#pragma unroll
      for (int j = 0; j < 4; ++j) {  // a channel of two keys in one register
        const uint32_t a0 = __byte_perm(x[0][j], x[1][j], 0x5410u);
        const uint32_t a1 = __byte_perm(x[0][j], x[1][j], 0x7632u);
        const uint32_t a2 = __byte_perm(x[2][j], x[3][j], 0x5410u);
        const uint32_t a3 = __byte_perm(x[2][j], x[3][j], 0x7632u);
        mma_16x8x16(o[i][j], a0, a1, a2, a3, w0, w1);
      }
    }
  }

  // the warps' results meet in shared memory
  float2* ml = reinterpret_cast<float2*>(sm + warps * heads * PR_DH);
  l += __shfl_xor_sync(0xffffffffu, l, 1);
  l += __shfl_xor_sync(0xffffffffu, l, 2);
  if (warp0 < chunks) m = fmaxf(m, KEYS_SEEN);
  if (c == 0 && n < heads) ml[warp * heads + n] = make_float2(m, l);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (2 * c + k >= heads) break;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float4* to = reinterpret_cast<float4*>(sm + (warp * heads + 2 * c + k) * PR_DH + i * 64 + n * 8);
      to[0] = make_float4(o[i][0][k], o[i][0][k + 2], o[i][1][k], o[i][1][k + 2]);
      to[1] = make_float4(o[i][2][k], o[i][2][k + 2], o[i][3][k], o[i][3][k + 2]);
    }
  }
  __syncthreads();
  for (int g = warp; g < heads; g += warps) {
    Joined x;
    for (int w = 0; w < warps; ++w) x.add(ml[w * heads + g], sm + (w * heads + g) * PR_DH, lane);
    if (a.cluster == 1) {
      x.store(a, t, head0 + g, lane);
    } else {  // the CTA's result where its first warp's was
      reinterpret_cast<float4*>(sm + g * PR_DH)[lane] = x.o;
      __syncwarp();
      if (lane == 0) ml[g] = make_float2(x.m, x.l);
    }
  }
  if (a.cluster == 1) return;
  cluster_sync_all();
  for (int g = rank + warp * a.cluster; g < heads; g += warps * a.cluster) {
    Joined x;
    for (int r = 0; r < a.cluster; ++r) x.add_peer(smem_u32(ml + g), smem_u32(sm + g * PR_DH), r, lane);
    x.store(a, t, head0 + g, lane);
  }
  cluster_sync_all();  // no CTA leaves while another reads its shared memory
}

}  // namespace

// Groups of the query heads of a key head, PR_HEADS at most in each.
static int rows_groups(int H, int Hkv) { return (H / Hkv + PR_HEADS - 1) / PR_HEADS; }

// CTAs for a row and group of heads: several, a cluster, where that leaves none of
// them waiting for a place, and 128 keys for each. Of 152 SMs, clusters of eight (and
// of seven) find 120 to be resident on at once, of six 132, of five, four and three
// 135: 2,000 keys of 15 rows take 7.1 us with eight, 8.1 with six, of 16 rows 12.4
// and 8.2; of 45 rows 13.6 with two, 11.9 with three, 17.5 with four.
static int rows_cluster(int64_t units, int64_t keys) {
  const int sms = num_sms();
  if (keys >= 1024 && units * 8 <= sms * 4 / 5) return 8;
  if (keys >= 768 && units * 6 <= sms * 7 / 8) return 6;
  for (int n = 5; n >= 3; --n)
    if (keys >= 128 * n && units * n <= sms * 8 / 9) return n;
  return keys >= 256 && units * 2 <= sms ? 2 : 1;
}

// Whether rows are taken one by one: `keys` is what a row can see at most, the room in
// its table and the prefix (how many it sees is known on the device only). Measured with
// tables as wide as the sequences are long, against the tensor-core kernel, us (here /
// there; it takes 11, 73, 235 and 963 where the tables of 1 row of 250 keys, 64 of 256,
// 42 heads, 1,024 of 256, 32 on 8, and 16,384 of 64, 8 on 2, have room for more, this one
// 5, 65, 173 and 193):
//   a CTA or a cluster per row and group of heads, all at once: one row, 4 heads, 250
//     keys 5.3 / 10.7, 1,000 keys 5.6 / 13.2, 8,000 keys 13.1 / 15.7, 12,000 keys
//     17.9 / 16.8; 84 CTAs of 4,000 keys in pairs 24 / 27; 126 CTAs of 2,000 keys
//     26 / 35; 16 rows of one sequence, 1,000 keys, 12 heads on 4: 8.3 / 14.8
//   more CTAs than SMs (a row's keys are read for itself, and once more per group of
//     its heads): 1,024 rows of 256 keys, 32 heads on 8: 175 / 250; 96 rows of up to
//     1,000 keys: 50 / 54, of 1,000 keys 83 / 74, of 2,000 keys 157 / 130; 512 rows of
//     1,000 keys, 16 heads on 1: 74 / 61, of 60 keys 9 / 28. Several rows of one
//     sequence read its keys several times: 8 sequences of 64 rows and keys, 4 heads
//     8.5 / 10.5, 2 of 40 rows and 500 keys 17 / 13. So does every row a prefix, where
//     the other kernel takes longer too: 32 rows of 42 heads behind 100 keys, 120 of
//     their own 32 / 36, behind 900 keys 90 / 49
bool paged_rows_fit(int T, int H, int Hkv, int B, int64_t keys, int prefix_len) {
  const int64_t groups = rows_groups(H, Hkv), units = groups * T * Hkv, sms = num_sms();
  if (units <= sms) return keys <= std::min(2048 * rows_cluster(units, keys), 10240);
  if (keys * groups * groups > 1024) return false;
  if (prefix_len > 0) return units * keys <= 2048 * sms;
  return T <= B || units * keys <= 900 * sms;
}

h3_status launch_paged_rows(const void* q, int64_t ld_q, void* o, int64_t ld_o, int H, float scale,
                            bool causal, const void* k_cache, const void* v_cache, int Hkv,
                            const PagedBatch& batch, const int32_t* prefix_pages, int prefix_len,
                            float* part_o, float* part_ml, cudaStream_t s) {
  RowsArgs a{};
  a.b = batch;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k_cache);
  a.v = static_cast<const __nv_bfloat16*>(v_cache);
  a.o = static_cast<__nv_bfloat16*>(o);
  a.ld_q = ld_q;
  a.ld_o = ld_o;
  a.Hkv = Hkv;
  a.G = H / Hkv;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.causal = causal ? 1 : 0;
  a.prefix_pages = prefix_pages;
  a.prefix_len = prefix_len;
  a.part_o = part_o;
  a.part_ml = part_ml;
  const int64_t keys = (static_cast<int64_t>(batch.max_pages) << batch.page_log2) + prefix_len;
  a.groups = rows_groups(H, Hkv);
  a.sets = a.groups * Hkv;
  const int64_t units = static_cast<int64_t>(batch.T) * a.sets;
  const int sms = num_sms(), chunks = static_cast<int>((keys + PR_CHUNK - 1) / PR_CHUNK);
  const bool many = units > 4 * sms;
  a.cluster = rows_cluster(units, keys);
  const int row = std::min(a.G, PR_HEADS) * (PR_DH * 4 + 8);  // a warp's results
  // where CTAs take turns, fewer warps for few keys: less to join, more CTAs per SM
  // (16,384 rows of 64 keys, 8 heads on 2: one warp 210 us, two 221, four 304; 1,024
  // rows of 1,000 keys, 32 on 8: four 344, two 352, one 417)
  int warps = many ? std::min((chunks + 7) / 8, 4) : PR_MAX_WARPS;
  warps = std::max(std::min(warps, chunks), 1);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(units * a.cluster));
  cfg.blockDim = dim3(32 * warps);
  cfg.dynamicSmemBytes = static_cast<size_t>(warps) * row;
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = a.cluster;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = a.cluster > 1 ? 1 : 0;
  const cudaError_t e = units <= sms ? cudaLaunchKernelEx(&cfg, paged_rows_kernel<1>, a)
                                     : cudaLaunchKernelEx(&cfg, paged_rows_kernel<2>, a);
  return cuda_fail(e, "paged attention of rows: launch");
}

}  // namespace h3
