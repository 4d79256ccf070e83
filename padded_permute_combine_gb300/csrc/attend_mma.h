// The kernel of the decode attention of bf16 caches, on the tensor cores
// (attention_decode.cu has the whole of it), and its launches.
#pragma once

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

// Sizes of a variant: DP elements of a row for a warp (64 or 128), TEAM warps that
// share the row, HEADS query heads at a time (8 or 16), BY: bytes that rows are aligned to and multiples of (16, 4 or 2).
template <int DP, int HEADS, int BY, int TEAM> struct Mma {
  static constexpr bool SHIFT = BY == 2;
  static constexpr int kWarps = DP == 128 ? (HEADS == 8 ? 8 : 12) : (SHIFT ? 12 : 16) / TEAM * TEAM;
  // Pieces of a row are swizzled by its number, or rows are one piece further apart: no two rows' pieces in one bank.
  static constexpr int kPitch = DP * 2 + (SHIFT ? 16 : 0);
  static constexpr int kStageBytes = 2 * kTile * kPitch;
  static constexpr int kStages = DP == 128 && HEADS == 16 ? 2 : 3;  // 162 to 192 KB an SM
  static constexpr int kScores = HEADS / 2;  // of a lane
  static constexpr size_t kRings = (size_t)kWarps * kStages * kStageBytes;
  static constexpr size_t kSmem = kRings + (TEAM > 1 ? (size_t)2 * kWarps * kWarp * kScores * 4 : 0);
};

// S = Q K^T and O += P V by m16n8k16 products: the query heads of a kv head are
// the rows, 16 keys a step. Decoding has few rows, so the products are never
// the bound (16 keys of 128 elements: 32 to 48 instructions in the 350 clocks
// that the SM's share of HBM needs for them). P goes in as two bf16 numbers, the
// second what the first one's rounding left; with eight heads or fewer the
// second takes the rows that they leave empty, and costs nothing.
// Rows are copied in pieces of 16 bytes, or of 4 where they are off 16. Rows off 4
// (SHIFT) are copied as the aligned pieces of 16 that hold them (a piece that
// holds an element lies inside the element's allocation) and moved into place in
// shared memory, piece by piece, when they have come.
// What takes longer than its bytes do is bound by the latency of a warp's
// instructions, eight warps an SM with rows of 128 elements. So the warps of a
// team share the rows, 64 elements each: they copy, multiply and sum their own
// columns, twice as many warps on an SM, and meet once a tile to add up the
// scores, of which each has a part.
template <int DP, int HEADS, int BY, int TEAM>
__global__ void __launch_bounds__(Mma<DP, HEADS, BY, TEAM>::kWarps * kWarp, 1) attend_mma_kernel(const AttendArgs a) {
  using S = Mma<DP, HEADS, BY, TEAM>;
  constexpr bool SHIFT = S::SHIFT;
  constexpr int kWarps = S::kWarps, kStages = S::kStages, kPitch = S::kPitch;
  constexpr int kTurns = DP / 32;  // of four lanes over the 16-byte pieces of a row
  constexpr int kSteps = DP / 16;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int s_prefix[kWarps * kWarp], s_warp[kWarps];
  __shared__ unsigned s_mask[kWarps][kStages][SHIFT ? 2 : 1];  // rows that are there: all 16 or, with SHIFT, eight and eight
  __shared__ uint8_t s_low[kWarps][SHIFT ? kStages : 1][kTile];  // rows' offsets to 16 bytes
  const int lane = lane_id(), warp = threadIdx.x / kWarp, team = warp / TEAM, rank = warp - team * TEAM;
  const int col0 = rank * DP, D = min(DP, a.D - col0);  // the warp's columns
  const uint32_t ring = smem_u32(smem) + warp * kStages * S::kStageBytes;
  if (SHIFT || D < DP) {  // pieces behind D are never copied, and have to be numbers
    uint4* z = reinterpret_cast<uint4*>(smem + (size_t)warp * kStages * S::kStageBytes);
    for (int i = lane; i < kStages * S::kStageBytes / 16; i += kWarp) z[i] = make_uint4(0, 0, 0, 0);
  }
  await_previous_kernel();
  start_next_kernel();
  Share share;
  Cursor in;
  const int count = my_range(a, team, kWarps / TEAM, s_prefix, s_warp, share, in);
  if (count == 0) return;
  const int r = share.r, kv = share.hv / a.parts, part = share.hv - kv * a.parts;
  __syncwarp();
  char* const keys = a.k + 2 * col0;
  char* const values = a.v + 2 * col0;
  const int h0 = kv * a.group + part * HEADS, heads = min(HEADS, a.group - part * HEADS);

  // Copies of a tile: K then V, 16 rows each, whole rows at a time, so that each
  // fetch is one of 256 bytes (four lanes a row take 40 instructions instead of
  // 150, but pieces of 64 bytes: 64 ragged sequences 157 us instead of 147). With
  // SHIFT there are more instructions a copy, and four lanes a row win.
  Cursor at = in;
  constexpr int kPiece = SHIFT ? 16 : BY;  // bytes
  constexpr int kChunks = DP * 2 / kPiece, kRowsPass = kWarp / kChunks, kPasses = kTile / kRowsPass;
  const int r0 = lane & 7, quarter = lane >> 3, pieces = (2 * D + kPiece - 1) / kPiece;  // eight lanes that meet in shared memory have eight rows: eight banks
  const int chunk = lane % kChunks, sub = lane / kChunks;
  int issued = 0, page[2] = {page_entry(a, in, SHIFT ? r0 : lane & (kTile - 1)), SHIFT ? page_entry(a, in, r0 + 8) : 0};
  const intptr_t apart = values - keys;
  // Of a row's piece `chunk`: 16 bytes of it lie at their number ^ (row & 7).
  const auto place = [&](int row) { return row * kPitch + ((chunk * kPiece / 16) ^ (row & 7)) * 16 + chunk * kPiece % 16; };
  const auto issue = [&](bool look) {  // look: for the next tile's page
    if (issued < count) {
      const int stage = issued % kStages;
      const int fresh = in.fresh_row();  // the new token's
      const char* kn = a.k_new + in.b * a.kn_row + kv * a.kn_head + 2 * col0;
      const char* vn = a.v_new + in.b * a.vn_row + kv * a.vn_head + 2 * col0;
      if constexpr (SHIFT) {
        const uint32_t base = ring + stage * S::kStageBytes + r0 * kPitch + quarter * 16;
        int64_t new_at = -1;  // of the new token's row, in its lanes
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const int64_t off = row_offset(a, in, r0 + 8 * w, page[w], kv);
          const unsigned there = __ballot_sync(0xffffffffu, off >= 0);
          if (lane == 0) s_mask[warp][stage][w] = there & 0xffu;
          const int bytes = off >= 0 ? 16 : 0;
          const uint32_t to = base + 8 * w * kPitch;
          const uintptr_t k_from = reinterpret_cast<uintptr_t>(keys) + (off < 0 ? 0 : off), v_from = k_from + apart;
          // The aligned pieces from the row's first byte's on. A row that is not there is zero to its end.
          const int k_low = (int)(k_from & 15), v_low = (int)(v_from & 15);
          const int k_end = bytes == 0 ? 2 * DP + 16 : 2 * D + k_low, v_end = bytes == 0 ? 2 * DP + 16 : 2 * D + v_low;
          if (quarter == 0) s_low[warp][stage][r0 + 8 * w] = (uint8_t)(k_low | v_low << 4);
          if (fresh == r0 + 8 * w) new_at = off;
          if (off < 0 || r0 + 8 * w != fresh) {
            const char* kp = reinterpret_cast<const char*>(k_from - k_low) + quarter * 16;
            const char* vp = reinterpret_cast<const char*>(v_from - v_low) + quarter * 16;
#pragma unroll
            for (int i = 0; i <= kTurns; ++i) {
              if (i == kTurns && quarter != 0) continue;
              if (quarter * 16 + i * 64 < k_end) cp_async16(to + i * 64, kp + i * 64, bytes);
              if (quarter * 16 + i * 64 < v_end) cp_async16(to + i * 64 + kTile * kPitch, vp + i * 64, bytes);
            }
          }
        }
        if (fresh >= 0 && fresh < kTile) {  // the new token, by the whole warp, to where the row's own bytes would lie
          new_at = __shfl_sync(0xffffffffu, new_at, fresh & 7);
          if (new_at >= 0) {
            const uintptr_t k_to = reinterpret_cast<uintptr_t>(keys) + new_at, v_to = k_to + apart;
            unsigned char* row = smem + (size_t)warp * kStages * S::kStageBytes + stage * S::kStageBytes + fresh * kPitch;
            uint16_t kk[DP / kWarp], vv[DP / kWarp];
#pragma unroll
            for (int j = 0; j < DP / kWarp; ++j) {
              const int d = lane + j * kWarp;
              kk[j] = d < D ? reinterpret_cast<const uint16_t*>(kn)[d] : 0;
              vv[j] = d < D ? reinterpret_cast<const uint16_t*>(vn)[d] : 0;
            }
#pragma unroll
            for (int j = 0; j < DP / kWarp; ++j) {
              const int d = lane + j * kWarp;
              if (d >= D) continue;
              reinterpret_cast<uint16_t*>(row + (k_to & 15))[d] = kk[j];
              reinterpret_cast<uint16_t*>(row + kTile * kPitch + (v_to & 15))[d] = vv[j];
              if (part == 0) {
                reinterpret_cast<uint16_t*>(k_to)[d] = kk[j];
                reinterpret_cast<uint16_t*>(v_to)[d] = vv[j];
              }
            }
          }
        }
      } else {
        const int row = lane & (kTile - 1);
        int64_t off = row_offset(a, in, row, page[0], kv);
        const unsigned there = __ballot_sync(0xffffffffu, off >= 0) & 0xffffu;
        if (lane == 0) s_mask[warp][stage][0] = there;
        const uint32_t base = ring + stage * S::kStageBytes;
        if (fresh >= 0 && fresh < kTile && (there >> fresh & 1)) {
          const int64_t to = __shfl_sync(0xffffffffu, off, fresh);
          if (row == fresh) off = -2;
          if (sub == 0 && chunk < pieces) {
            const uint32_t dst = base + place(fresh);
            cp_async<kPiece>(dst, kn + chunk * kPiece, kPiece);
            cp_async<kPiece>(dst + kTile * kPitch, vn + chunk * kPiece, kPiece);
            if (part == 0) {
              using V = typename Vec<kPiece>::T;
              const V kk = *reinterpret_cast<const V*>(kn + chunk * kPiece), vv = *reinterpret_cast<const V*>(vn + chunk * kPiece);
              *reinterpret_cast<V*>(keys + to + chunk * kPiece) = kk;
              *reinterpret_cast<V*>(values + to + chunk * kPiece) = vv;
            }
          }
        }
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
          const int row_i = i * kRowsPass + sub;
          const int64_t from = __shfl_sync(0xffffffffu, off, row_i);
          if (from == -2 || chunk >= pieces) continue;
          const int bytes = from < 0 ? 0 : kPiece;
          const int64_t o = from < 0 ? 0 : from + chunk * kPiece;
          const uint32_t dst = base + place(row_i);
          cp_async<kPiece>(dst, keys + o, bytes);
          cp_async<kPiece>(dst + kTile * kPitch, values + o, bytes);
        }
      }
      if (++issued < count) {
        in.next(a);
        if (look) {
          page[0] = page_entry(a, in, SHIFT ? r0 : lane & (kTile - 1));
          if constexpr (SHIFT) page[1] = page_entry(a, in, r0 + 8);
        }
      }
    }
    cp_commit();
  };
  // SHIFT: moves a tile's rows to the beginnings of their places, zeros behind
  // D. In a turn the four lanes of a row take five pieces and put four.
  const auto align = [&](int stage) {
    int low[4];  // K of rows r0 and r0 + 8, V of them
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int both = s_low[warp][SHIFT ? stage : 0][r0 + 8 * w];
      low[w] = both & 15;
      low[2 + w] = both >> 4;
    }
    uint4* base = reinterpret_cast<uint4*>(smem + (ring - smem_u32(smem)) + stage * S::kStageBytes + r0 * kPitch + quarter * 16);
#pragma unroll 1
    for (int i = 0; i * 4 < pieces; ++i) {
      uint32_t v[4][4];
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint4* from = base + ((w & 1) * 8 * kPitch + (w >> 1) * kTile * kPitch) / 16 + i * 4;
        const uint4 x = from[0], y = from[1];
        // low / 4 words further on (by two, then by one), and two bytes more where it is odd in them.
        const bool two = low[w] & 8, one = low[w] & 4;
        const uint32_t w0 = two ? x.z : x.x, w1 = two ? x.w : x.y, w2 = two ? y.x : x.z, w3 = two ? y.y : x.w, w4 = two ? y.z : y.x,
                       w5 = two ? y.w : y.y;
        const uint32_t t0 = one ? w1 : w0, t1 = one ? w2 : w1, t2 = one ? w3 : w2, t3 = one ? w4 : w3, t4 = one ? w5 : w4;
        const int bits = (low[w] & 2) * 8;
        v[w][0] = __funnelshift_r(t0, t1, bits);
        v[w][1] = __funnelshift_r(t1, t2, bits);
        v[w][2] = __funnelshift_r(t2, t3, bits);
        v[w][3] = __funnelshift_r(t3, t4, bits);
      }
      const int left = D - 8 * (quarter + 4 * i);  // elements of the row from this piece on
      if (left < 8) {
#pragma unroll
        for (int w = 0; w < 4; ++w)
#pragma unroll
          for (int e = 0; e < 4; ++e) v[w][e] &= 2 * e + 2 <= left ? 0xffffffffu : 2 * e >= left ? 0u : 0xffffu;
      }
      __syncwarp();
#pragma unroll
      for (int w = 0; w < 4; ++w)
        base[((w & 1) * 8 * kPitch + (w >> 1) * kTile * kPitch) / 16 + i * 4] = make_uint4(v[w][0], v[w][1], v[w][2], v[w][3]);
    }
    __syncwarp();
  };
  {  // the first tiles' pages on their way together
    int first[kStages][2];
    Cursor ahead = in;
#pragma unroll
    for (int i = 1; i < kStages; ++i) {
      if (i >= count) continue;
      ahead.next(a);
      first[i][0] = page_entry(a, ahead, SHIFT ? r0 : lane & (kTile - 1));
      if constexpr (SHIFT) first[i][1] = page_entry(a, ahead, r0 + 8);
    }
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
      issue(false);
      page[0] = first[i + 1][0];
      if constexpr (SHIFT) page[1] = first[i + 1][1];
    }
  }

  uint32_t q[kSteps][4];
  float o[DP / 8][4], m[2], l[2];
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
      const char* rows = a.q + at.b * a.q_row + 2 * col0;
#pragma unroll
      for (int ks = 0; ks < kSteps; ++ks)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int h = g + (e & 1) * 8, d = ks * 16 + t * 2 + (e >> 1) * 8;
          const char* from = rows + (h0 + h) * a.q_head + d * 2;
          uint32_t x = 0;
          if (!((HEADS == 8 && (e & 1)) || h >= heads || d >= D)) {
            if constexpr (SHIFT) {
              x = __ldg(reinterpret_cast<const unsigned short*>(from));
              if (d + 1 < D) x |= (uint32_t)__ldg(reinterpret_cast<const unsigned short*>(from) + 1) << 16;
            } else {
              x = __ldg(reinterpret_cast<const unsigned*>(from));
            }
          }
          q[ks][e] = x;
        }
#pragma unroll
      for (int n = 0; n < DP / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][e] = 0.0f;
      m[0] = m[1] = -INFINITY;
      l[0] = l[1] = 0.0f;
    }
    cp_wait<kStages - 2>();
    __syncwarp();
    const int stage = i % kStages;
    const unsigned there = SHIFT ? s_mask[warp][stage][0] | s_mask[warp][stage][SHIFT ? 1 : 0] << 8 : s_mask[warp][stage][0];
    const bool all = there == 0xffffu;
    issue(true);  // into the stage that the previous tile left
    if constexpr (SHIFT) align(stage);
    const uint32_t base = ring + stage * S::kStageBytes;
    float s[2][4];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[n][e] = 0.0f;
#pragma unroll
    for (int ks = 0; ks < kSteps; ++ks) {
      if (SHIFT && ks * 16 >= D) continue;
      uint32_t b[4];
      ldmatrix(b, base + k_at + (((ks * 2 + (mi & 1)) ^ swizzle) * 16));
      mma(s[0], q[ks], b[0], b[1]);
      mma(s[1], q[ks], b[2], b[3]);
    }
    if constexpr (TEAM > 1) {
      // The scores' parts, added up in the same order by every warp. Two places in turn: who writes one again
      // has met, a tile earlier, those who read it.
      float* mine = reinterpret_cast<float*>(smem + S::kRings) + ((i & 1) * kWarps + team * TEAM) * kWarp * S::kScores + lane * 4;
      float part[S::kScores];
#pragma unroll
      for (int k = 0; k < S::kScores; ++k) part[k] = HEADS == 8 ? s[k / 2][k % 2] : s[k / 4 % 2][k % 4];
#pragma unroll
      for (int k = 0; k < S::kScores; k += 4)
        *reinterpret_cast<float4*>(mine + rank * kWarp * S::kScores + k * kWarp) = make_float4(part[k], part[k + 1], part[k + 2], part[k + 3]);
      asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "n"(TEAM * kWarp) : "memory");
#pragma unroll
      for (int k = 0; k < S::kScores; k += 4) {
        float4 sum = *reinterpret_cast<const float4*>(mine + k * kWarp);
#pragma unroll
        for (int w = 1; w < TEAM; ++w) {
          const float4 x = *reinterpret_cast<const float4*>(mine + w * kWarp * S::kScores + k * kWarp);
          sum.x += x.x;
          sum.y += x.y;
          sum.z += x.z;
          sum.w += x.w;
        }
        part[k] = sum.x;
        part[k + 1] = sum.y;
        part[k + 2] = sum.z;
        part[k + 3] = sum.w;
      }
#pragma unroll
      for (int k = 0; k < S::kScores; ++k) (HEADS == 8 ? s[k / 2][k % 2] : s[k / 4 % 2][k % 4]) = part[k];
    }
    uint32_t hi[4], lo2[4];
    constexpr int kRows = HEADS == 8 ? 1 : 2;  // rows g and g + 8
    float keep[2] = {1.0f, 1.0f};
    bool moved = false;
#pragma unroll
    for (int w = 0; w < kRows; ++w) {
      float top = -INFINITY;
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float& x = s[n][2 * w + e];
          x *= a.scale;
          if (!all && !(there >> (n * 8 + t * 2 + e) & 1)) x = -INFINITY;
          top = fmaxf(top, x);
        }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const float now = fmaxf(m[w], top), from = now == -INFINITY ? 0.0f : now;
      if (now > m[w]) {
        moved = true;
        keep[w] = ex2(m[w] - from);
        m[w] = now;
      }
      float sum = 0.0f;
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const float p0 = ex2(s[n][2 * w] - from), p1 = ex2(s[n][2 * w + 1] - from);
        sum += p0 + p1;
        const uint32_t h = pack_bf16x2(p0, p1);
        const uint32_t rest = pack_bf16x2(p0 - __uint_as_float(h << 16), p1 - __uint_as_float(h & 0xffff0000u));
        if constexpr (HEADS == 8) {
          hi[2 * n] = h;
          hi[2 * n + 1] = rest;
        } else {
          hi[2 * n + w] = h;
          lo2[2 * n + w] = rest;
        }
      }
      l[w] = l[w] * keep[w] + sum;
    }
    if (__any_sync(0xffffffffu, moved)) {
      if constexpr (HEADS == 8) keep[1] = keep[0];
#pragma unroll
      for (int n = 0; n < DP / 8; ++n) {
        if (SHIFT && n * 8 >= D) continue;
        o[n][0] *= keep[0];
        o[n][1] *= keep[0];
        o[n][2] *= keep[1];
        o[n][3] *= keep[1];
      }
    }
#pragma unroll
    for (int c = 0; c < kSteps; ++c) {
      if (SHIFT && c * 16 >= D) continue;
      uint32_t b[4];
      ldmatrix_trans(b, base + v_at + (((c * 2 + (mi >> 1)) ^ swizzle) * 16));
      mma(o[2 * c], hi, b[0], b[1]);
      mma(o[2 * c + 1], hi, b[2], b[3]);
      if constexpr (HEADS == 16) {
        mma(o[2 * c], lo2, b[0], b[1]);
        mma(o[2 * c + 1], lo2, b[2], b[3]);
      }
    }
    const bool last = at.tile == at.tiles - 1;
    if (last || i == count - 1) {
      const bool whole = last && first_tile == 0;
#pragma unroll
      for (int w = 0; w < kRows; ++w) {
        float sum = l[w];
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        const int h = g + w * 8;
        if (h >= heads) continue;
        const int64_t head = (whole ? (int64_t)at.b : (int64_t)r + at.b) * a.heads + h0 + h;
        const float inv = share_of(sum);
#pragma unroll
        for (int n = 0; n < DP / 8; ++n) {
          const int d = n * 8 + t * 2;
          if (d >= D) continue;
          float x = o[n][2 * w], y = o[n][2 * w + 1];
          if constexpr (HEADS == 8) {
            x += o[n][2];
            y += o[n][3];
          }
          __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + head * a.D + col0 + d;
          if constexpr (SHIFT) {  // D may be odd
            if (whole) {
              out[0] = __float2bfloat16_rn(x * inv);
              if (d + 1 < D) out[1] = __float2bfloat16_rn(y * inv);
            } else {
              a.part_o[head * a.D + col0 + d] = x;
              if (d + 1 < D) a.part_o[head * a.D + col0 + d + 1] = y;
            }
          } else if (whole) {
            *reinterpret_cast<uint32_t*>(out) = pack_bf16x2(x * inv, y * inv);
          } else {
            *reinterpret_cast<float2*>(a.part_o + head * a.D + col0 + d) = make_float2(x, y);
          }
        }
        if (t == 0 && rank == 0) {
          if (!whole) {
            a.part_ml[head] = make_float2(m[w], sum);
          } else if (a.lse != nullptr) {
            a.lse[head] = log_sum_of(m[w], sum);
          }
        }
      }
      fresh = true;
    }
    if (i + 1 < count) at.next(a);
  }
}

template <int DP, int HEADS, int BY, int TEAM> int launch_mma(AttendArgs& a, cudaStream_t s) {
  using S = Mma<DP, HEADS, BY, TEAM>;
  static std::atomic<bool> raised[kSmemDevices];
  auto k = attend_mma_kernel<DP, HEADS, BY, TEAM>;
  if (!allow_smem(k, raised)) return MOE_ERR_CUDA;
  cut(a, HEADS, S::kWarps / TEAM);
  launch(k, dim3(ctas_of(a, S::kWarps / TEAM)), dim3(S::kWarps * kWarp), S::kSmem, s, a);
  return check_launch();
}
template <int DP, int BY, int TEAM> int launch_mma_heads(AttendArgs& a, cudaStream_t s) {
  return a.group <= 8 ? launch_mma<DP, 8, BY, TEAM>(a, s) : launch_mma<DP, 16, BY, TEAM>(a, s);
}
template <int BY> int launch_mma_dim(AttendArgs& a, cudaStream_t s) {
  // Aligned rows of up to 128 elements are one warp's: 64 ragged sequences 147 us, with teams of two 151.
  if constexpr (BY == 16)
    if (a.D > 64 && a.D <= 128) return launch_mma_heads<128, BY, 1>(a, s);
  if constexpr (BY != 16)
    if (a.D > 64 && a.D <= 128) return launch_mma_heads<64, BY, 2>(a, s);
  return a.D <= 64 ? launch_mma_heads<64, BY, 1>(a, s) : a.D <= 192 ? launch_mma_heads<64, BY, 3>(a, s) : launch_mma_heads<64, BY, 4>(a, s);
}

}  // namespace
}  // namespace moe
