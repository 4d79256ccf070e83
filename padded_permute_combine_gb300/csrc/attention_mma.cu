// Decode attention of bf16 caches, on the tensor cores (attention_decode.cu has the whole of it).
#include "attend.h"

namespace moe {
namespace {

__device__ __forceinline__ void ldmatrix(uint32_t (&f)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(f[0]), "=r"(f[1]), "=r"(f[2]), "=r"(f[3]) : "r"(at));
}
__device__ __forceinline__ void ldmatrix_trans(uint32_t (&f)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(f[0]), "=r"(f[1]), "=r"(f[2]), "=r"(f[3]) : "r"(at));
}
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Sizes of a variant: DP elements of a padded row (64, 128 or 256), MT tiles of
// 16 query heads (0: eight heads in one), SHIFT for rows off 16 bytes.
template <int DP, int MT, bool SHIFT> struct Mma {
  static constexpr int kHeads = MT == 0 ? 8 : 16 * MT, kTiles = MT == 0 ? 1 : MT;
  static constexpr int kWarps = DP == 256 ? 4 : 8;
  // Pieces of a row are swizzled by its number, or rows are one piece further apart: no two rows' pieces in one bank.
  static constexpr int kPitch = DP * 2 + (SHIFT ? 16 : 0);
  static constexpr int kStageBytes = 2 * kTile * kPitch;
  static constexpr int kStages = DP == 64 ? 6 : 3;  // 192 to 221 KB an SM
  static constexpr size_t kSmem = (size_t)kWarps * kStages * kStageBytes;
};

// S = Q K^T and O += P V by m16n8k16 products: the query heads of a kv head are
// the rows, 16 keys a step. Decoding has few rows, so the products are never
// the bound (16 keys of 128 elements: 32 to 48 instructions in the 350 clocks
// that the SM's share of HBM needs for them). P goes in as two bf16 numbers, the
// second what the first one's rounding left; with eight heads or fewer the
// second takes the rows that they leave empty, and costs nothing.
// Rows off 16 bytes (SHIFT) are copied as the aligned pieces that hold them (a
// piece that holds an element lies inside the element's allocation) and moved
// into place in shared memory, piece by piece, when they have come.
template <int DP, int MT, bool SHIFT>
__global__ void __launch_bounds__(Mma<DP, MT, SHIFT>::kWarps * kWarp, 1) attend_mma_kernel(const AttendArgs a) {
  using S = Mma<DP, MT, SHIFT>;
  constexpr int kWarps = S::kWarps, kStages = S::kStages, kTiles = S::kTiles, kPitch = S::kPitch;
  constexpr int kChunks = DP / 8, kRowsPass = kWarp / kChunks, kPasses = kTile / kRowsPass;  // 16-byte pieces of a row
  constexpr int kSteps = DP / 16;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int s_prefix[kWarps * kWarp], s_warp[kWarps];
  __shared__ unsigned s_mask[kWarps][kStages];
  __shared__ uint64_t s_low[kWarps][SHIFT ? kStages : 1];  // four bits a row: its offset to 16 bytes
  await_previous_kernel();
  start_next_kernel();
  const int lane = lane_id(), warp = threadIdx.x / kWarp;
  const int total = line_prefix(a, s_prefix, s_warp);
  const int HV = a.kv_heads * a.parts, gw = blockIdx.x * kWarps + warp;
  const int r = gw / HV, hv = gw - r * HV, kv = hv / a.parts, part = hv - kv * a.parts;
  if (total == 0) return;
  const int ranges = ranges_of(a, total);
  if (r >= ranges) return;
  const int lo = range_begin(r, ranges, total), count = range_begin(r + 1, ranges, total) - lo;
  if (count <= 0) return;
  const int D = a.D, h0 = kv * a.group + part * S::kHeads, heads = min(S::kHeads, a.group - part * S::kHeads);
  const uint32_t ring = smem_u32(smem) + warp * kStages * S::kStageBytes;
  if (SHIFT || D < DP) {  // pieces behind D are never copied, and have to be numbers
    uint4* z = reinterpret_cast<uint4*>(smem + (size_t)warp * kStages * S::kStageBytes);
    for (int i = lane; i < kStages * S::kStageBytes / 16; i += kWarp) z[i] = make_uint4(0, 0, 0, 0);
    __syncwarp();
  }
  const auto place = [](int row, int c) { return row * kPitch + (SHIFT ? c : c ^ (row & 7)) * 16; };

  // Copies of a tile: K then V, 16 rows each.
  Cursor in = find_tile(a, s_prefix, lo);
  Cursor at = in;
  int issued = 0, page = page_entry(a, in, lane & (kTile - 1));
  const int chunk = lane % kChunks, sub = lane / kChunks;
  const bool copies = chunk * 8 < D;
  const int k_low = SHIFT ? (int)(reinterpret_cast<uintptr_t>(a.k) & 15) : 0, v_low = SHIFT ? (int)(reinterpret_cast<uintptr_t>(a.v) & 15) : 0;
  const auto issue = [&]() {
    if (issued < count) {
      const int stage = issued % kStages, row = lane & (kTile - 1);
      int64_t off = row_offset(a, in, row, page, kv);
      const unsigned valid = __ballot_sync(0xffffffffu, off >= 0) & 0xffffu;
      if (lane == 0) s_mask[warp][stage] = valid;
      if constexpr (SHIFT) {
        uint64_t low = lane < kTile ? (uint64_t)(off & 15) << (4 * row) : 0;
#pragma unroll
        for (int d = 1; d < kTile; d <<= 1) low |= __shfl_xor_sync(0xffffffffu, low, d);
        if (lane == 0) s_low[warp][stage] = low;
      }
      const int fresh = a.k_new != nullptr ? in.n - 1 - (in.first + in.tile * kTile) : -1;  // the new token's row
      const uint32_t base = ring + stage * S::kStageBytes;
      if (fresh >= 0 && fresh < kTile && (valid >> fresh & 1)) {
        const int64_t to = __shfl_sync(0xffffffffu, off, fresh);
        if (row == fresh) off = -2;
        const char* kn = a.k_new + in.b * a.kn_row + kv * a.kn_head;
        const char* vn = a.v_new + in.b * a.vn_row + kv * a.vn_head;
        if constexpr (SHIFT) {  // to where the row's own bytes would lie
          unsigned char* k_to = smem + (size_t)warp * kStages * S::kStageBytes + stage * S::kStageBytes + fresh * kPitch;
          unsigned char* v_to = k_to + kTile * kPitch + ((to + v_low) & 15);
          k_to += (to + k_low) & 15;
          for (int d = lane; d < D; d += kWarp) {
            const uint16_t kk = reinterpret_cast<const uint16_t*>(kn)[d], vv = reinterpret_cast<const uint16_t*>(vn)[d];
            reinterpret_cast<uint16_t*>(k_to)[d] = kk;
            reinterpret_cast<uint16_t*>(v_to)[d] = vv;
            if (part == 0) {
              reinterpret_cast<uint16_t*>(a.k + to)[d] = kk;
              reinterpret_cast<uint16_t*>(a.v + to)[d] = vv;
            }
          }
        } else if (sub == 0 && copies) {
          const uint32_t dst = base + place(fresh, chunk);
          cp_async16(dst, kn + chunk * 16, 16);
          cp_async16(dst + kTile * kPitch, vn + chunk * 16, 16);
          if (part == 0) {
            *reinterpret_cast<uint4*>(a.k + to + chunk * 16) = *reinterpret_cast<const uint4*>(kn + chunk * 16);
            *reinterpret_cast<uint4*>(a.v + to + chunk * 16) = *reinterpret_cast<const uint4*>(vn + chunk * 16);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        const int row_i = i * kRowsPass + sub;
        const int64_t from = __shfl_sync(0xffffffffu, off, row_i);
        if (from == -2) continue;
        const uint32_t dst = base + place(row_i, chunk);
        if constexpr (SHIFT) {
          // The pieces from the row's first byte's on; with an offset there may be one more than the row has.
          const char* k_from = a.k + (from < 0 ? -k_low : from);
          const char* v_from = a.v + (from < 0 ? -v_low : from);
          const int k_off = (int)(reinterpret_cast<uintptr_t>(k_from) & 15), v_off = (int)(reinterpret_cast<uintptr_t>(v_from) & 15);
          const int bytes = from < 0 ? 0 : 16;
#pragma unroll
          for (int c = chunk; c <= kChunks; c += kChunks) {
            if (from < 0 || c * 16 < 2 * D + k_off) cp_async16(dst + (c - chunk) * 16, k_from - k_off + c * 16, bytes);
            if (from < 0 || c * 16 < 2 * D + v_off) cp_async16(dst + (c - chunk) * 16 + kTile * kPitch, v_from - v_off + c * 16, bytes);
          }
        } else if (copies) {
          const int bytes = from < 0 ? 0 : 16;
          const int64_t o = from < 0 ? 0 : from + chunk * 16;
          cp_async16(dst, a.k + o, bytes);
          cp_async16(dst + kTile * kPitch, a.v + o, bytes);
        }
      }
      if (++issued < count) {
        in.next(a);
        page = page_entry(a, in, row);
      }
    }
    cp_commit();
  };
  // SHIFT: moves a tile's rows to the beginnings of their places, zeros behind D.
  const auto align = [&](int stage) {
    const uint64_t low = s_low[warp][SHIFT ? stage : 0];
    unsigned char* base = smem + (size_t)warp * kStages * S::kStageBytes + stage * S::kStageBytes;
#pragma unroll
    for (int i = 0; i < 2 * kPasses; ++i) {
      const int row = (i % kPasses) * kRowsPass + sub, off = ((int)(low >> (4 * row)) + (i < kPasses ? k_low : v_low)) & 15;
      uint4* to = reinterpret_cast<uint4*>(base + (i < kPasses ? 0 : kTile * kPitch) + row * kPitch) + chunk;
      const uint4 x = to[0], y = to[1];
      const int left = 2 * (D - 8 * chunk);  // bytes of the row from this piece on
      // off / 4 words further on (by two, then by one), and two bytes more where it is odd in them.
      const bool two = off & 8, one = off & 4;
      const uint32_t w0 = two ? x.z : x.x, w1 = two ? x.w : x.y, w2 = two ? y.x : x.z, w3 = two ? y.y : x.w, w4 = two ? y.z : y.x,
                     w5 = two ? y.w : y.y;
      const uint32_t t0 = one ? w1 : w0, t1 = one ? w2 : w1, t2 = one ? w3 : w2, t3 = one ? w4 : w3, t4 = one ? w5 : w4;
      const int bits = (off & 2) * 8;
      uint32_t v[4] = {__funnelshift_r(t0, t1, bits), __funnelshift_r(t1, t2, bits), __funnelshift_r(t2, t3, bits), __funnelshift_r(t3, t4, bits)};
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = left >= 4 * e + 4 ? v[e] : left <= 4 * e ? 0u : v[e] & 0xffffu;
      __syncwarp();
      to[0] = make_uint4(v[0], v[1], v[2], v[3]);
    }
    __syncwarp();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue();

  uint32_t q[kTiles][kSteps][4];
  float o[kTiles][DP / 8][4], m[kTiles][2], l[kTiles][2];
  const int g = lane >> 2, t = lane & 3;
  const int mi = lane >> 3, lr = lane & 7;
  const int swizzle = SHIFT ? 0 : lr;
  const uint32_t k_at = ((mi >> 1) * 8 + lr) * kPitch, v_at = ((mi & 1) * 8 + lr) * kPitch + kTile * kPitch;
  bool fresh = true;
  int first_tile = at.tile;
  for (int i = 0; i < count; ++i) {
    if (fresh) {
      fresh = false;
      first_tile = at.tile;
      const char* rows = a.q + at.b * a.q_row;
#pragma unroll
      for (int u = 0; u < kTiles; ++u) {
#pragma unroll
        for (int ks = 0; ks < kSteps; ++ks)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int h = u * 16 + g + (e & 1) * 8, d = ks * 16 + t * 2 + (e >> 1) * 8;
            const char* from = rows + (h0 + h) * a.q_head + d * 2;
            uint32_t x = 0;
            if (!((MT == 0 && (e & 1)) || h >= heads || d >= D)) {
              if constexpr (SHIFT) {
                x = __ldg(reinterpret_cast<const unsigned short*>(from));
                if (d + 1 < D) x |= (uint32_t)__ldg(reinterpret_cast<const unsigned short*>(from) + 1) << 16;
              } else {
                x = __ldg(reinterpret_cast<const unsigned*>(from));
              }
            }
            q[u][ks][e] = x;
          }
#pragma unroll
        for (int n = 0; n < DP / 8; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[u][n][e] = 0.0f;
        m[u][0] = m[u][1] = -INFINITY;
        l[u][0] = l[u][1] = 0.0f;
      }
    }
    cp_wait<kStages - 2>();
    __syncwarp();
    const int stage = i % kStages;
    const unsigned valid = s_mask[warp][stage];
    issue();  // into the stage that the previous tile left
    if constexpr (SHIFT) align(stage);
    const uint32_t base = ring + stage * S::kStageBytes;
    float s[kTiles][2][4];
#pragma unroll
    for (int u = 0; u < kTiles; ++u)
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[u][n][e] = 0.0f;
#pragma unroll
    for (int ks = 0; ks < kSteps; ++ks) {
      uint32_t b[4];
      ldmatrix(b, base + k_at + (((ks * 2 + (mi & 1)) ^ swizzle) * 16));
#pragma unroll
      for (int u = 0; u < kTiles; ++u) {
        mma(s[u][0], q[u][ks], b[0], b[1]);
        mma(s[u][1], q[u][ks], b[2], b[3]);
      }
    }
    uint32_t hi[kTiles][4], lo2[kTiles][4];
#pragma unroll
    for (int u = 0; u < kTiles; ++u) {
      constexpr int kRows = MT == 0 ? 1 : 2;  // rows g and g + 8
      float keep[2] = {1.0f, 1.0f};
      bool moved = false;
#pragma unroll
      for (int w = 0; w < kRows; ++w) {
        float top = -INFINITY;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float& x = s[u][n][2 * w + e];
            x *= a.scale;
            if (valid != 0xffffu && !(valid >> (n * 8 + t * 2 + e) & 1)) x = -INFINITY;
            top = fmaxf(top, x);
          }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const float now = fmaxf(m[u][w], top), from = now == -INFINITY ? 0.0f : now;
        if (now > m[u][w]) {
          moved = true;
          keep[w] = ex2(m[u][w] - from);
          m[u][w] = now;
        }
        float sum = 0.0f;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const float p0 = ex2(s[u][n][2 * w] - from), p1 = ex2(s[u][n][2 * w + 1] - from);
          sum += p0 + p1;
          const uint32_t h = pack_bf16x2(p0, p1);
          const uint32_t rest = pack_bf16x2(p0 - __uint_as_float(h << 16), p1 - __uint_as_float(h & 0xffff0000u));
          if constexpr (MT == 0) {
            hi[u][2 * n] = h;
            hi[u][2 * n + 1] = rest;
          } else {
            hi[u][2 * n + w] = h;
            lo2[u][2 * n + w] = rest;
          }
        }
        l[u][w] = l[u][w] * keep[w] + sum;
      }
      if (__any_sync(0xffffffffu, moved)) {
        if constexpr (MT == 0) keep[1] = keep[0];
#pragma unroll
        for (int n = 0; n < DP / 8; ++n) {
          o[u][n][0] *= keep[0];
          o[u][n][1] *= keep[0];
          o[u][n][2] *= keep[1];
          o[u][n][3] *= keep[1];
        }
      }
    }
#pragma unroll
    for (int c = 0; c < kSteps; ++c) {
      uint32_t b[4];
      ldmatrix_trans(b, base + v_at + (((c * 2 + (mi >> 1)) ^ swizzle) * 16));
#pragma unroll
      for (int u = 0; u < kTiles; ++u) {
        mma(o[u][2 * c], hi[u], b[0], b[1]);
        mma(o[u][2 * c + 1], hi[u], b[2], b[3]);
        if constexpr (MT > 0) {
          mma(o[u][2 * c], lo2[u], b[0], b[1]);
          mma(o[u][2 * c + 1], lo2[u], b[2], b[3]);
        }
      }
    }
    const bool last = at.tile == at.tiles - 1;
    if (last || i == count - 1) {
      const bool whole = last && first_tile == 0;
#pragma unroll
      for (int u = 0; u < kTiles; ++u)
#pragma unroll
        for (int w = 0; w < (MT == 0 ? 1 : 2); ++w) {
          float sum = l[u][w];
          sum += __shfl_xor_sync(0xffffffffu, sum, 1);
          sum += __shfl_xor_sync(0xffffffffu, sum, 2);
          const int h = u * 16 + g + w * 8;
          if (h >= heads) continue;
          const int64_t head = (whole ? (int64_t)at.b : (int64_t)r + at.b) * a.heads + h0 + h;
          const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
          for (int n = 0; n < DP / 8; ++n) {
            const int d = n * 8 + t * 2;
            if (d >= D) continue;
            float x = o[u][n][2 * w], y = o[u][n][2 * w + 1];
            if constexpr (MT == 0) {
              x += o[u][n][2];
              y += o[u][n][3];
            }
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + head * D + d;
            if constexpr (SHIFT) {  // D may be odd
              if (whole) {
                out[0] = __float2bfloat16_rn(x * inv);
                if (d + 1 < D) out[1] = __float2bfloat16_rn(y * inv);
              } else {
                a.part_o[head * D + d] = x;
                if (d + 1 < D) a.part_o[head * D + d + 1] = y;
              }
            } else if (whole) {
              *reinterpret_cast<uint32_t*>(out) = pack_bf16x2(x * inv, y * inv);
            } else {
              *reinterpret_cast<float2*>(a.part_o + head * D + d) = make_float2(x, y);
            }
          }
          if (t == 0) {
            if (!whole) {
              a.part_ml[head] = make_float2(m[u][w], sum);
            } else if (a.lse != nullptr) {
              a.lse[head] = sum > 0.0f ? (m[u][w] + log2f(sum)) * kLn2 : -INFINITY;
            }
          }
        }
      fresh = true;
    }
    if (i + 1 < count) at.next(a);
  }
}

template <int DP, int MT, bool SHIFT> int launch_mma(AttendArgs& a, cudaStream_t s) {
  using S = Mma<DP, MT, SHIFT>;
  static std::atomic<bool> raised[kSmemDevices];
  auto k = attend_mma_kernel<DP, MT, SHIFT>;
  if (!allow_smem(k, raised)) return MOE_ERR_CUDA;
  cut(a, S::kHeads, S::kWarps);
  launch(k, dim3(ctas_of(a, S::kWarps)), dim3(S::kWarps * kWarp), S::kSmem, s, a);
  return check_launch();
}
template <int DP, bool SHIFT> int launch_mma_heads(AttendArgs& a, cudaStream_t s) {
  if (a.group <= 8) return launch_mma<DP, 0, SHIFT>(a, s);
  if constexpr (DP < 256 && !SHIFT)  // two tiles of heads at once: the registers hold them up to 128 elements
    if (a.group > 16) return launch_mma<DP, 2, SHIFT>(a, s);
  return launch_mma<DP, 1, SHIFT>(a, s);
}
template <bool SHIFT> int launch_mma_dim(AttendArgs& a, cudaStream_t s) {
  return a.D <= 64 ? launch_mma_heads<64, SHIFT>(a, s) : a.D <= 128 ? launch_mma_heads<128, SHIFT>(a, s) : launch_mma_heads<256, SHIFT>(a, s);
}

}  // namespace

int attend_mma(AttendArgs& a, bool pieces, cudaStream_t s) { return pieces ? launch_mma_dim<false>(a, s) : launch_mma_dim<true>(a, s); }

}  // namespace moe
