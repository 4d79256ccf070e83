// Decode attention of fp32 caches (attention_decode.cu has the whole of it).
#include "attend.h"
#include "vec_math.cuh"

namespace moe {
namespace {

// A row in shared memory: pieces of 16 bytes, a multiple of four of them. The
// lanes that read two neighbouring keys at once find them in different banks:
// rows of an odd multiple of 64 bytes do so by themselves, in others the odd
// keys' pieces are exchanged in groups of four.
struct RowPieces {
  int pieces, pitch, swap;
  __host__ __device__ explicit RowPieces(int D) : pieces((D + 3) / 4), pitch((pieces + 3) / 4 * 4), swap(pitch % 8 == 0 ? 4 : 0) {}
};
// Warps of an SM, as registers and shared memory allow: twelve with rows of up to some 80 elements.
template <int GM, int NC> constexpr int kSmWarps = GM <= 4 && NC == 1 ? 12 : 8;
constexpr int kSlots = 3;  // of a warp's ring, a tile's keys or values each

__device__ __forceinline__ uint64_t pair(float a, float b) { return f2_pack(__float_as_uint(a), __float_as_uint(b)); }

// A warp takes a tile's 16 keys, then its values, through a ring of three slots:
// while one is used the next two are on their way. Scores: lane (key, quarter)
// takes the fourth of the pieces of two keys that `quarter` says, for all GM
// heads; values: a lane owns pieces of the rows for all heads. Two elements an
// instruction (fma.f32x2). VB: bytes of an asynchronous copy, 4 where rows are
// off 16.
template <int GM, int NC, int VB>
__global__ void __launch_bounds__(kSmWarps<GM, NC> * kWarp, 1) attend_rows_kernel(const AttendArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int s_prefix[kSmWarps<GM, NC> * kWarp], s_warp[kSmWarps<GM, NC>];
  const int lane = lane_id(), warp = threadIdx.x / kWarp, warps = blockDim.x / kWarp;
  const int D = a.D;
  const RowPieces row(D);
  const int slot_bytes = kTile * row.pitch * 16;
  unsigned char* own = smem + (size_t)warp * (kSlots * slot_bytes + GM * row.pitch * 16 + GM * kTile * 8);
  float* qs = reinterpret_cast<float*>(own + kSlots * slot_bytes);
  uint64_t* ps = reinterpret_cast<uint64_t*>(qs + GM * row.pitch * 4);  // [GM][16], each probability twice
  const uint32_t ring = smem_u32(own);
  // What lies behind D in a row's last piece stays zero, and the query rows of heads behind the group.
  for (int i = (VB == 16 ? kSlots * slot_bytes / 16 : 0) + lane; i < (kSlots * slot_bytes + GM * row.pitch * 16) / 16; i += kWarp)
    reinterpret_cast<uint4*>(own)[i] = make_uint4(0, 0, 0, 0);
  await_previous_kernel();
  start_next_kernel();
  Share share;
  Cursor in;
  const int count = my_range(a, warp, warps, s_prefix, s_warp, share, in);
  if (count == 0) return;
  const int r = share.r, kv = share.hv / a.parts, part = share.hv - kv * a.parts;
  __syncwarp();

  // Copies of a tile's keys, then of its values: four lanes a row (rows r0 and
  // r0 + 8), so that a copy's addresses are a register and a constant.
  constexpr int kTurns = NC * 8;  // of the four lanes over a row
  Cursor at = in;
  const int r0 = lane >> 2, part4 = lane & 3, pieces = row.pieces;
  int issued = 0, slot_in = 0, page[2] = {page_entry(a, in, r0), page_entry(a, in, r0 + 8)}, bytes[2];
  unsigned there[2];  // rows of the tile issued last that are there, four equal bits each
  const char* from[2];
  const intptr_t apart = a.v - a.k;
  const int flip = r0 & 1 ? row.swap * 16 : 0;
  const uint32_t place = r0 * row.pitch * 16 + part4 * VB;
  const auto issue = [&](bool values) {
    if (issued < count) {
      const uint32_t base = ring + slot_in * slot_bytes + place;
      const int fresh = in.fresh_row();  // the new token's
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        if (!values) {
          const int64_t off = row_offset(a, in, r0 + 8 * w, page[w], kv);
          there[w] = __ballot_sync(0xffffffffu, off >= 0);
          bytes[w] = off >= 0 ? VB : 0;
          from[w] = a.k + (off < 0 ? 0 : off);
        }
        const char* src = from[w] + (values ? apart : 0);
        if (r0 + 8 * w == fresh && bytes[w] != 0)
          src = values ? a.v_new + in.b * a.vn_row + kv * a.vn_head : a.k_new + in.b * a.kn_row + kv * a.kn_head;
        if constexpr (VB == 16) {
          src += part4 * VB;
          const uint32_t to = base + 8 * w * row.pitch * 16, even = to + flip, odd = to - flip;  // 64 bytes on in every other 64
#pragma unroll
          for (int i = 0; i < kTurns; ++i) {
            if (part4 + 4 * i >= pieces) continue;
            cp_async16((i & 1 ? odd : even) + i * 64, src + i * 64, bytes[w]);
          }
        } else {  // a row at a time, 32 words side by side
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint64_t row_at = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(src), 4 * i);
            const int n = __shfl_sync(0xffffffffu, bytes[w], 4 * i);
            const uint32_t to = ring + slot_in * slot_bytes + (8 * w + i) * row.pitch * 16;
#pragma unroll
            for (int j = 0; j < 4 * NC; ++j) {
              const int d = lane + j * kWarp;
              if (d < D) cp_async4(to + ((d >> 2) ^ (i & 1 ? row.swap : 0)) * 16 + (d & 3) * 4, reinterpret_cast<const char*>(row_at) + d * 4, n);
            }
          }
        }
      }
      if (!values && part == 0 && fresh >= 0 && fresh < kTile) {
        // The new token into the cache, by the whole warp while the tile is on its way (by the row's four
        // lanes, in front of the copies: one sequence of 600 tokens 14.2 us instead of 9.5, 16 of 4000 95 instead of 85).
        const int row_lane = fresh % 8 * 4;
        float* k_to = reinterpret_cast<float*>(__shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(fresh < 8 ? from[0] : from[1]), row_lane));
        if (__shfl_sync(0xffffffffu, fresh < 8 ? bytes[0] : bytes[1], row_lane) != 0) {
          float* v_to = k_to + apart / 4;
          const float* kn = reinterpret_cast<const float*>(a.k_new + in.b * a.kn_row + kv * a.kn_head);
          const float* vn = reinterpret_cast<const float*>(a.v_new + in.b * a.vn_row + kv * a.vn_head);
          float kk[4 * NC], vv[4 * NC];
#pragma unroll
          for (int j = 0; j < 4 * NC; ++j) {
            const int d = lane + j * kWarp;
            kk[j] = d < D ? kn[d] : 0.0f;
            vv[j] = d < D ? vn[d] : 0.0f;
          }
#pragma unroll
          for (int j = 0; j < 4 * NC; ++j) {
            const int d = lane + j * kWarp;
            if (d >= D) continue;
            k_to[d] = kk[j];
            v_to[d] = vv[j];
          }
        }
      }
      if (values && ++issued < count) {
        in.next(a);
        page[0] = page_entry(a, in, r0);
        page[1] = page_entry(a, in, r0 + 8);
      }
      slot_in = slot_in == kSlots - 1 ? 0 : slot_in + 1;
    }
    cp_commit();
  };
  issue(false);
  issue(true);

  const int h0 = kv * a.group + part * GM, heads = min(GM, a.group - part * GM);
  const int key = lane >> 2, quarter = lane & 3, swap = key & 1 ? row.swap : 0;
  float m[GM], l[GM];
  uint64_t o[GM][NC][2];
  bool fresh = true;
  int first_tile = at.tile, slot = 0;
  for (int i = 0; i < count; ++i) {
    if (fresh) {
      fresh = false;
      first_tile = at.tile;
      for (int h = 0; h < heads; ++h) {
        const float* q = reinterpret_cast<const float*>(a.q + at.b * a.q_row + (h0 + h) * a.q_head);
        for (int d = lane; d < D; d += kWarp) qs[h * row.pitch * 4 + d] = q[d] * a.scale;
      }
#pragma unroll
      for (int h = 0; h < GM; ++h) {
        m[h] = -INFINITY;
        l[h] = 0.0f;
#pragma unroll
        for (int j = 0; j < NC; ++j) o[h][j][0] = o[h][j][1] = 0;
      }
    }
    cp_wait<1>();
    __syncwarp();
    const unsigned now_there[2] = {there[0], there[1]};  // no later tile's keys are issued yet
    issue(false);      // into the slot that the previous tile's values left
    {
      // Scores of two keys, all heads, the same in the four lanes of a key.
      const ulonglong2* ks = reinterpret_cast<const ulonglong2*>(own + slot * slot_bytes) + key * row.pitch;
      uint64_t s[GM][2];
#pragma unroll
      for (int h = 0; h < GM; ++h) s[h][0] = s[h][1] = 0;
#pragma unroll 2
      for (int p = quarter; p < row.pieces; p += 4) {
        const ulonglong2 k0 = ks[p ^ swap], k1 = ks[8 * row.pitch + (p ^ swap)];  // pairs of elements
#pragma unroll
        for (int h = 0; h < GM; ++h) {
          const ulonglong2 qq = reinterpret_cast<const ulonglong2*>(qs)[h * row.pitch + p];
          s[h][0] = f2_fma(qq.y, k0.y, f2_fma(qq.x, k0.x, s[h][0]));
          s[h][1] = f2_fma(qq.y, k1.y, f2_fma(qq.x, k1.x, s[h][1]));
        }
      }
#pragma unroll
      for (int h = 0; h < GM; ++h) {
        float x[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float lo2, hi2;
          f2_unpack(s[h][e], lo2, hi2);
          x[e] = lo2 + hi2;
          x[e] += __shfl_xor_sync(0xffffffffu, x[e], 1);
          x[e] += __shfl_xor_sync(0xffffffffu, x[e], 2);
          if (!(now_there[e] >> (4 * key) & 1)) x[e] = -INFINITY;
        }
        float t = fmaxf(x[0], x[1]);
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
        const float now = fmaxf(m[h], t), from = now == -INFINITY ? 0.0f : now;
        if (now > m[h]) {  // the same in every lane
          const float keep = exp2f(m[h] - from);
          m[h] = now;
          l[h] *= keep;
#pragma unroll
          for (int j = 0; j < NC; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) o[h][j][e] = f2_mul(o[h][j][e], pair(keep, keep));
        }
        const float p0 = exp2f(x[0] - from), p1 = exp2f(x[1] - from);
        l[h] += p0 + p1;  // four lanes have each
        if (quarter == 0) {
          ps[h * kTile + key] = pair(p0, p0);
          ps[h * kTile + key + 8] = pair(p1, p1);
        }
      }
    }
    slot = slot == kSlots - 1 ? 0 : slot + 1;
    cp_wait<1>();
    __syncwarp();
    issue(true);
    {
      const ulonglong2* vs = reinterpret_cast<const ulonglong2*>(own + slot * slot_bytes);
#pragma unroll 4
      for (int e = 0; e < kTile; e += 2) {
        ulonglong2 pr[GM];  // the probabilities of two keys, each twice
#pragma unroll
        for (int h = 0; h < GM; ++h) pr[h] = *reinterpret_cast<const ulonglong2*>(ps + h * kTile + e);
#pragma unroll
        for (int j = 0; j < NC; ++j) {
          const int p = lane + j * kWarp;
          if (p >= row.pieces) continue;
          const ulonglong2 v0 = vs[e * row.pitch + p], v1 = vs[(e + 1) * row.pitch + (p ^ row.swap)];
#pragma unroll
          for (int h = 0; h < GM; ++h) {
            o[h][j][0] = f2_fma(pr[h].y, v1.x, f2_fma(pr[h].x, v0.x, o[h][j][0]));
            o[h][j][1] = f2_fma(pr[h].y, v1.y, f2_fma(pr[h].x, v0.y, o[h][j][1]));
          }
        }
      }
    }
    slot = slot == kSlots - 1 ? 0 : slot + 1;
    const bool last = at.tile == at.tiles - 1;
    if (last || i == count - 1) {
      const bool whole = last && first_tile == 0;
#pragma unroll
      for (int h = 0; h < GM; ++h) {
        float sum = l[h];
#pragma unroll
        for (int d = 4; d < kWarp; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (h >= heads) continue;
        const int64_t head = (whole ? (int64_t)at.b : (int64_t)r + at.b) * a.heads + h0 + h;
        const float inv = whole ? share_of(sum) : 1.0f;
        float* to = (whole ? static_cast<float*>(a.out) : a.part_o) + head * D;
#pragma unroll
        for (int j = 0; j < NC; ++j) {
          float v[4];
          f2_unpack(o[h][j][0], v[0], v[1]);
          f2_unpack(o[h][j][1], v[2], v[3]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int d = 4 * (lane + j * kWarp) + e;
            if (d < D) to[d] = v[e] * inv;
          }
        }
        if (lane == 0) {
          if (!whole) {
            a.part_ml[head] = make_float2(m[h], sum);
          } else if (a.lse != nullptr) {
            a.lse[head] = log_sum_of(m[h], sum);
          }
        }
      }
      fresh = true;
      __syncwarp();  // the next query comes into the same place
    }
    if (i + 1 < count) at.next(a);
  }
}

template <int GM, int NC, int VB> int launch_rows(AttendArgs& a, cudaStream_t s) {
  static std::atomic<bool> raised[kSmemDevices];
  auto k = attend_rows_kernel<GM, NC, VB>;
  if (!allow_smem(k, raised)) return MOE_ERR_CUDA;
  const RowPieces row(a.D);
  const int bytes = kSlots * kTile * row.pitch * 16 + GM * row.pitch * 16 + GM * kTile * 8;  // of a warp
  const int fit = 224 * 1024 / bytes, warps = fit < kSmWarps<GM, NC> ? fit : kSmWarps<GM, NC>;
  cut(a, GM, warps);
  launch(k, dim3(ctas_of(a, warps)), dim3(warps * kWarp), (size_t)warps * bytes, s, a);
  return check_launch();
}
template <int GM, int VB> int launch_rows_dim(AttendArgs& a, cudaStream_t s) {
  return a.D <= 128 ? launch_rows<GM, 1, VB>(a, s) : launch_rows<GM, 2, VB>(a, s);
}
template <int VB> int launch_rows_heads(AttendArgs& a, cudaStream_t s) {
  return a.group <= 2 ? launch_rows_dim<2, VB>(a, s) : a.group <= 4 ? launch_rows_dim<4, VB>(a, s) : launch_rows_dim<8, VB>(a, s);
}

}  // namespace

int attend_rows(AttendArgs& a, bool pieces, cudaStream_t s) { return pieces ? launch_rows_heads<16>(a, s) : launch_rows_heads<4>(a, s); }

}  // namespace moe
