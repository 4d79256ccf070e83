// Decode attention of fp32 caches (attention_decode.cu has the whole of it).
#include "attend.h"

namespace moe {
namespace {

constexpr int kKeys = 8;  // of a step

// A row in shared memory: pieces of 16 bytes, a multiple of four of them. The
// lanes that read two neighbouring keys at once find them in different banks:
// rows of an odd multiple of 64 bytes do so by themselves, in others the odd
// keys' pieces are exchanged in groups of four.
struct RowPieces {
  int pieces, pitch, swap;
  __host__ __device__ explicit RowPieces(int D) : pieces((D + 3) / 4), pitch((pieces + 3) / 4 * 4), swap(pitch % 8 == 0 ? 4 : 0) {}
};

// A warp takes 8 keys at a time through a ring of kStages of them. Scores: lane
// (key, quarter) takes the fourth of the key's pieces that `quarter` says, for
// all GM heads; values: a lane owns pieces of the rows for all heads. VB: bytes
// of an asynchronous copy, 4 where rows are off 16.
template <int GM, int NC, int VB, int kStages>
__global__ void __launch_bounds__(kSmWarps * kWarp, 1) attend_rows_kernel(const AttendArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int s_prefix[kSmWarps * kWarp], s_warp[kSmWarps];
  __shared__ unsigned s_mask[kSmWarps][kStages];
  await_previous_kernel();
  start_next_kernel();
  const int lane = lane_id(), warp = threadIdx.x / kWarp, warps = blockDim.x / kWarp;
  const int total = line_prefix(a, s_prefix, s_warp);
  const int HV = a.kv_heads * a.parts, gw = blockIdx.x * warps + warp;
  const int r = gw / HV, hv = gw - r * HV, kv = hv / a.parts, part = hv - kv * a.parts;
  if (total == 0) return;
  const int ranges = ranges_of(a, total);
  if (r >= ranges) return;
  const int lo = range_begin(r, ranges, total), count = 2 * (range_begin(r + 1, ranges, total) - lo);  // steps
  if (count <= 0) return;

  const int D = a.D;
  const RowPieces row(D);
  const int half_bytes = kKeys * row.pitch * 16, stage_bytes = 2 * half_bytes;
  unsigned char* own = smem + (size_t)warp * (kStages * stage_bytes + GM * row.pitch * 16 + GM * kKeys * 4);
  float* qs = reinterpret_cast<float*>(own + kStages * stage_bytes);
  float* ps = qs + GM * row.pitch * 4;
  const uint32_t ring = smem_u32(own);
  for (int i = lane; i < (kStages * stage_bytes + GM * row.pitch * 16) / 16; i += kWarp)  // what lies behind D stays zero
    reinterpret_cast<uint4*>(own)[i] = make_uint4(0, 0, 0, 0);
  __syncwarp();

  // Copies of a step: 8 rows of keys, then of values.
  Cursor in = find_tile(a, s_prefix, lo);
  Cursor at = in;
  int issued = 0, page = page_entry(a, in, lane & (kTile - 1));
  int64_t off = -1;
  unsigned valid = 0;
  const int copies = VB == 16 ? row.pieces : D;  // of a row
  const auto issue = [&]() {
    if (issued < count) {
      const int stage = issued % kStages, part8 = issued & 1, mine = lane & (kTile - 1);
      if (part8 == 0) {
        off = row_offset(a, in, mine, page, kv);
        valid = __ballot_sync(0xffffffffu, off >= 0) & 0xffffu;
      }
      if (lane == 0) s_mask[warp][stage] = valid >> (part8 * kKeys) & 0xffu;
      const int fresh = a.k_new != nullptr ? in.n - 1 - (in.first + in.tile * kTile) - part8 * kKeys : -1;  // the new token's row
      const uint32_t base = ring + stage * stage_bytes;
#pragma unroll
      for (int i = 0; i < kKeys; ++i) {
        const int64_t from = __shfl_sync(0xffffffffu, off, part8 * kKeys + i);
        if (from < 0) {
          // A row that is not there: zeros, which its probability of zero can be multiplied by.
          for (int c = lane; c < row.pieces; c += kWarp) {
            uint4* dst = reinterpret_cast<uint4*>(own + stage * stage_bytes) + i * row.pitch + (c ^ (i & 1 ? row.swap : 0));
            dst[0] = dst[kKeys * row.pitch] = make_uint4(0, 0, 0, 0);
          }
          continue;
        }
        const char* ksrc = a.k + from;
        const char* vsrc = a.v + from;
        if (i == fresh) {
          ksrc = a.k_new + in.b * a.kn_row + kv * a.kn_head;
          vsrc = a.v_new + in.b * a.vn_row + kv * a.vn_head;
          if (part == 0)
            for (int d = lane; d < D; d += kWarp) {
              reinterpret_cast<float*>(a.k + from)[d] = reinterpret_cast<const float*>(ksrc)[d];
              reinterpret_cast<float*>(a.v + from)[d] = reinterpret_cast<const float*>(vsrc)[d];
            }
        }
        for (int c = lane; c < copies; c += kWarp) {
          if constexpr (VB == 16) {
            const uint32_t dst = base + (i * row.pitch + (c ^ (i & 1 ? row.swap : 0))) * 16;
            cp_async16(dst, ksrc + c * 16, 16);
            cp_async16(dst + half_bytes, vsrc + c * 16, 16);
          } else {
            const uint32_t dst = base + (i * row.pitch + ((c >> 2) ^ (i & 1 ? row.swap : 0))) * 16 + (c & 3) * 4;
            cp_async4(dst, ksrc + c * 4, 4);
            cp_async4(dst + half_bytes, vsrc + c * 4, 4);
          }
        }
      }
      if (++issued < count && part8 == 1) {
        in.next(a);
        page = page_entry(a, in, mine);
      }
    }
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue();

  const int h0 = kv * a.group + part * GM, heads = min(GM, a.group - part * GM);
  const int key = lane >> 2, quarter = lane & 3, swap = key & 1 ? row.swap : 0;
  float m[GM], l[GM], o[GM][NC][4];
  bool fresh = true;
  int first_tile = at.tile;
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
        for (int j = 0; j < NC; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[h][j][e] = 0.0f;
      }
    }
    cp_wait<kStages - 2>();
    __syncwarp();
    const int stage = i % kStages;
    const unsigned bits = s_mask[warp][stage];
    issue();  // into the stage that the previous step left
    const float4* ks = reinterpret_cast<const float4*>(own + stage * stage_bytes);
    const float4* vs = ks + kKeys * row.pitch;
    if (bits != 0) {
      // Scores of (key, all heads), the same in the four lanes of a key.
      float s[GM];
#pragma unroll
      for (int h = 0; h < GM; ++h) s[h] = 0.0f;
#pragma unroll 4
      for (int p = quarter; p < row.pieces; p += 4) {
        const float4 kk = ks[key * row.pitch + (p ^ swap)];
#pragma unroll
        for (int h = 0; h < GM; ++h) {
          const float4 qq = reinterpret_cast<const float4*>(qs)[h * row.pitch + p];
          s[h] = fmaf(qq.x, kk.x, fmaf(qq.y, kk.y, fmaf(qq.z, kk.z, fmaf(qq.w, kk.w, s[h]))));
        }
      }
#pragma unroll
      for (int h = 0; h < GM; ++h) {
        s[h] += __shfl_xor_sync(0xffffffffu, s[h], 1);
        s[h] += __shfl_xor_sync(0xffffffffu, s[h], 2);
        if (!(bits >> key & 1)) s[h] = -INFINITY;
        float t = s[h];
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
        const float now = fmaxf(m[h], t), base = now == -INFINITY ? 0.0f : now;
        if (now > m[h]) {  // the same in every lane
          const float keep = exp2f(m[h] - base);
          m[h] = now;
          l[h] *= keep;
#pragma unroll
          for (int j = 0; j < NC; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[h][j][e] *= keep;
        }
        const float pr = exp2f(s[h] - base);
        if (quarter == 0) {
          l[h] += pr;
          ps[h * kKeys + key] = pr;
        }
      }
      __syncwarp();
      float pr[GM][kKeys];
#pragma unroll
      for (int h = 0; h < GM; ++h)
#pragma unroll
        for (int e = 0; e < kKeys; e += 4) {
          const float4 x = *reinterpret_cast<const float4*>(ps + h * kKeys + e);
          pr[h][e] = x.x;
          pr[h][e + 1] = x.y;
          pr[h][e + 2] = x.z;
          pr[h][e + 3] = x.w;
        }
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        const int p = lane + j * kWarp;
        if (p < row.pieces) {
#pragma unroll
          for (int e = 0; e < kKeys; ++e) {
            const float4 vv = vs[e * row.pitch + (p ^ (e & 1 ? row.swap : 0))];
#pragma unroll
            for (int h = 0; h < GM; ++h) {
              o[h][j][0] = fmaf(pr[h][e], vv.x, o[h][j][0]);
              o[h][j][1] = fmaf(pr[h][e], vv.y, o[h][j][1]);
              o[h][j][2] = fmaf(pr[h][e], vv.z, o[h][j][2]);
              o[h][j][3] = fmaf(pr[h][e], vv.w, o[h][j][3]);
            }
          }
        }
      }
    }
    if ((i & 1) == 0) continue;
    const bool last = at.tile == at.tiles - 1;
    if (last || i == count - 1) {
      const bool whole = last && first_tile == 0;
#pragma unroll
      for (int h = 0; h < GM; ++h) {
        float sum = l[h];
#pragma unroll
        for (int d = 1; d < kWarp; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (h >= heads) continue;
        const int64_t head = (whole ? (int64_t)at.b : (int64_t)r + at.b) * a.heads + h0 + h;
        const float inv = whole ? (sum > 0.0f ? 1.0f / sum : 0.0f) : 1.0f;
        float* to = (whole ? static_cast<float*>(a.out) : a.part_o) + head * D;
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int d = 4 * (lane + j * kWarp) + e;
            if (d < D) to[d] = o[h][j][e] * inv;
          }
        if (lane == 0) {
          if (!whole) {
            a.part_ml[head] = make_float2(m[h], sum);
          } else if (a.lse != nullptr) {
            a.lse[head] = sum > 0.0f ? (m[h] + log2f(sum)) * kLn2 : -INFINITY;
          }
        }
      }
      fresh = true;
    }
    if (i + 1 < count) at.next(a);
  }
}

template <int GM, int NC, int VB, int kStages> int launch_rows(AttendArgs& a, int warps, size_t smem, cudaStream_t s) {
  static std::atomic<bool> raised[kSmemDevices];
  auto k = attend_rows_kernel<GM, NC, VB, kStages>;
  if (!allow_smem(k, raised)) return MOE_ERR_CUDA;
  cut(a, GM, warps);
  launch(k, dim3(ctas_of(a, warps)), dim3(warps * kWarp), smem, s, a);
  return check_launch();
}
template <int GM, int VB> int launch_rows_dim(AttendArgs& a, cudaStream_t s) {
  constexpr int kStages = GM == 8 ? 2 : 3;  // eight heads' rows need the room of the third
  const RowPieces row(a.D);
  const auto bytes = [&](int stages) { return (size_t)2 * stages * kKeys * row.pitch * 16 + GM * row.pitch * 16 + GM * kKeys * 4; };
  if (a.D <= 128) return launch_rows<GM, 1, VB, kStages>(a, 8, 8 * bytes(kStages), s);
  return launch_rows<GM, 2, VB, 2>(a, 5, 5 * bytes(2), s);
}
template <int VB> int launch_rows_heads(AttendArgs& a, cudaStream_t s) {
  return a.group <= 2 ? launch_rows_dim<2, VB>(a, s) : a.group <= 4 ? launch_rows_dim<4, VB>(a, s) : launch_rows_dim<8, VB>(a, s);
}

}  // namespace

int attend_rows(AttendArgs& a, bool pieces, cudaStream_t s) { return pieces ? launch_rows_heads<16>(a, s) : launch_rows_heads<4>(a, s); }

}  // namespace moe
