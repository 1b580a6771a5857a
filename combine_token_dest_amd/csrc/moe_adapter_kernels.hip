// gfx950 kernels of a shared projection with low-rank adapters:
//   y[r] = W x[r] + s_a B_a (A_a x[r]), a = ids[r].
//
// low_kernel makes the scaled low-rank values s_a A_a x: 1 or 8 rows of x to
// a workgroup, and the rows of A of each adapter that they name, one adapter
// after another.  Up to kLowFew rows share k between workgroups, whose float32
// sums the second kernel adds in turn.
//
// The shared product is that of moe_gemm_device.h.  Behind it, while the sums
// are still in registers, a wave goes through the adapters that its rows name,
// one after another: B_a's rows times the low values by matrix instructions,
// added to the rows that have this adapter and to no others (a row's result
// never meets another adapter's B, whatever is in it).  (Before the product it
// would wait no longer than the first tiles do, but the compiler then finds no
// registers for the product's loop.)
// The low values go in as three bfloat16 each, float32's 24 bits.  An infinity
// on either side meets all of the other's parts, of which none may be 0 or of
// the other sign then: low_parts() and the float16 path see to it.  Few rows
// take the kernel that streams the weights (moe_few_device.h), where each
// result adds its own adapter's sum over the rank in float32, made while the
// first weights are on their way.
//
// 2048 rows of 4096 x 7168 with five adapters of rank 16 take 144 us: 15 for the
// low values and the rest for the product, which alone takes 113; one row 4 and 11.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "moe_dense_internal.h"
#include "moe_few_device.h"
#include "moe_gemm_device.h"

namespace moe_ep_detail {
namespace {

// Eight elements from k on of COUNT rows of `rank`, which start `row` bytes
// after base; zeros past the rank.  All loads go out at once: with a branch
// for each row's end every load would wait for the one before.
template <int COUNT>
__device__ __forceinline__ void b_elements(const uint16_t* base, const uint32_t (&row)[COUNT], int k, int rank,
                                           u32x4 (&v)[COUNT]) {
  const uint8_t* p = reinterpret_cast<const uint8_t*>(base);
  if (rank >= 8) {
    // the last eight of the row where fewer are left, moved to the front
    const int have = rank - k, at = min(k, rank - 8) * 2;
#pragma unroll
    for (int i = 0; i < COUNT; ++i) v[i] = load_any8(p + (row[i] + at));
#pragma unroll
    for (int i = 0; i < COUNT; ++i) v[i] = keep_last(v[i], have);
  } else {
#pragma unroll
    for (int i = 0; i < COUNT; ++i) {
      const uint16_t* r = reinterpret_cast<const uint16_t*>(p + row[i]);
      uint32_t e[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) e[j] = r[min(k + j, rank - 1)];
#pragma unroll
      for (int j = 0; j < 8; ++j) e[j] = k + j < rank ? e[j] : 0u;
      v[i] = u32x4{e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16};
    }
  }
}

// A low value's parts (split_parts), where a part that would be 0 beside a
// number is 2^-40 of it instead: less than float32's 24 bits tell, and an
// infinity in B times each part has the number's sign.  (Numbers below 2^-100,
// beside which bfloat16 has no room for that, keep the zeros.)
__device__ __forceinline__ void low_parts(float v, uint16_t (&part)[kParts]) {
  split_parts(v, part);
  const int first = part[0], exponent = first >> 7 & 0xFF;
  const uint16_t least = (uint16_t)((first & 0x8000) | max(exponent - 40, 1) << 7);
#pragma unroll
  for (int pl = 1; pl < kParts; ++pl)
    if (exponent >= 27 && exponent < 255 && !(part[pl] & 0x7FFF)) part[pl] = least;
}

// split_f16 with a second part of 0 beside an infinity or NaN.
__device__ __forceinline__ void split_f16_finite(const u32x4& v, u32x4* hi, u32x4* lo) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = F16::to_float((uint16_t)v[i]), b = F16::to_float((uint16_t)(v[i] >> 16));
    const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b) & 0xFFFF0000u;
    float ra = a - __uint_as_float(ua & 0xFFFF0000u), rb = b - __uint_as_float(ub);
    ra = ra == ra ? ra : 0.0f;
    rb = rb == rb ? rb : 0.0f;
    (*hi)[i] = ua >> 16 | ub;
    (*lo)[i] = __float_as_uint(ra) >> 16 | (__float_as_uint(rb) & 0xFFFF0000u);
  }
}

// Eight bfloat16 with zeros for infinities and NaN.
__device__ __forceinline__ u32x4 finite_ones(const u32x4& v) {
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // an exponent of ones carries into its half's top bit, which then fills the half
    const uint32_t bad = ((v[i] & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
    r[i] = v[i] & ~((bad << 1) - (bad >> 15));
  }
  return r;
}
__device__ __forceinline__ bool all_finite(const u32x4& v) {
  uint32_t bad = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) bad |= (v[i] & 0x7F807F80u) + 0x00800080u;
  return !(bad & 0x80008000u);
}

constexpr int kLowWaves = 8;
// Calls of up to this many rows, which may be one request's each, take them
// one by one; more are prompts, whose rows share adapters.  (The host does not
// see the ids.)  Calls of 2048 columns, us, row by row and 8 rows at a time:
//                        an adapter a row           four prompts
//   k, rank     rows  128      512      1024     128      512      1024
//   2048, 16        18 28    25 35    49 56     18 18    19 18    33 29
//   7168, 16        34 61    52 73    98 115    30 30    44 41    79 68
//   4096, 64        36 48    70 72   130 147    27 22    44 33    77 54
//   7168, 128       72 82   172 190  343 352    49 35    96 60   172 95
constexpr int kLowSingle = 512;

// One pass of low_kernel: M adapters' rows of A with the workgroup's rows of x.
template <class T, int BLOCK, int RT, bool FEW, int M>
__device__ __forceinline__ void low_pass(const AdapterKArgs& a, const int (&ad)[M], int id, char* lds) {
  typedef Few<T, RT * M, 1, kLowWaves> F;
  static_assert(F::kLds >= RT * M * 1024, "the sums fit a wave's piece");
  f32x4 (*sums)[RT * M][16][4] = reinterpret_cast<f32x4 (*)[RT * M][16][4]>(lds);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, i = lane & 15;
  const int r0 = blockIdx.x * BLOCK, k0 = blockIdx.y * (16 * RT), split = blockIdx.z;
  const int R = a.rank, n = a.x.rows;
  // this part's steps of 64 k
  constexpr int splits = FEW ? kLowSplits : 1;
  const int steps = a.k / 64, left = a.k % 64;
  const int first = (int)((int64_t)steps * split / splits), last = (int)((int64_t)steps * (split + 1) / splits);
  F few;
  few.aim([&](int m, int r) { return a.a + ((int64_t)ad[m / RT] * R + min(k0 + m % RT * 16 + r, R - 1)) * a.k; },
          [&](int, int r) { return a.x.p + (int64_t)min(r0 + min(r, BLOCK - 1), n - 1) * a.x.stride; }, first,
          last - first, blockIdx.x, lds + wave * F::kLds);
  few.prime(wave, kLowWaves);
  f32x4 acc[RT * M][1] = {};
  few.run(wave, kLowWaves, acc);
  if (left && split == splits - 1 && wave == kLowWaves - 1) few.tail(left, acc);
  __syncthreads();                                        // the waves' pieces of lds become the sums
#pragma unroll
  for (int m = 0; m < RT * M; ++m) sums[wave][m][i][lane >> 4] = acc[m][0];
  __syncthreads();
  const float* sum = reinterpret_cast<const float*>(lds);
  // the last of the rank is followed by zeros up to the stride
  constexpr int kWide = RT == 1 && !FEW ? 32 : 16 * RT;
  const bool last_of_rank = k0 + 16 * RT >= R;
#pragma unroll
  for (int m = 0; m < M; ++m) {
    const float scale = a.scales ? a.scales[ad[m]] : 1.0f;
    for (int o = threadIdx.x; o < BLOCK * kWide; o += kLowWaves * 64) {
      const int r = o / kWide, c = o % kWide, k = k0 + c;
      float v = 0;
      if (c < 16 * RT) {
#pragma unroll
        for (int w = 0; w < kLowWaves; ++w) v += sum[((w * RT * M + m * RT + c / 16) * 16 + r) * 16 + c % 16];
      }
      v = k < R ? v * scale : 0.0f;
      if (__shfl(id, r) != ad[m] || k >= a.low_stride || (c >= 16 * RT && !last_of_rank)) continue;
      const int64_t at = (int64_t)(r0 + r) * a.low_stride + k, plane = (int64_t)n * a.low_stride;
      if constexpr (FEW) {
        static_cast<float*>(a.low)[split * plane + at] = v;
      } else {
        uint16_t part[kParts];
        low_parts(v, part);
#pragma unroll
        for (int pl = 0; pl < kParts; ++pl) static_cast<uint16_t*>(a.low)[pl * plane + at] = part[pl];
      }
    }
  }
  __syncthreads();
}

// The low values of BLOCK rows of x and 16 RT of the rank.
template <class T, int BLOCK, int RT, bool FEW>
__global__ void __launch_bounds__(kLowWaves * 64) low_kernel(AdapterKArgs a) {
  // two adapters a pass, where rows of two prompts meet
  constexpr bool kPairs = BLOCK > 1 && RT == 1;
  __shared__ __attribute__((aligned(1024))) char lds[kLowWaves * Few<T, kPairs ? 2 : RT, 1, kLowWaves>::kLds];
  const int row = blockIdx.x * BLOCK + min((int)threadIdx.x & 15, BLOCK - 1);
  // lanes of the same row name the same adapter; rows past the last none
  int id = row < a.x.rows ? a.ids[row] : -1;
  if (id < 0 || id >= a.adapters) id = -1;
  uint64_t pending = __ballot(id >= 0);
  auto next = [&]() {
    const int ad = __builtin_amdgcn_readlane(id, __builtin_ctzll(pending));
    pending &= ~__ballot(id == ad);
    return ad;
  };
  while (pending) {
    const int one[1] = {next()};
    if constexpr (kPairs) {
      if (pending) {
        const int two[2] = {one[0], next()};
        low_pass<T, BLOCK, RT, FEW, 2>(a, two, id, lds);
        continue;
      }
    }
    low_pass<T, BLOCK, RT, FEW, 1>(a, one, id, lds);
  }
}

// Up to 16 NT rows: 16 columns of the result to a workgroup.
template <class T, int NT, int WAVES>
__global__ void __launch_bounds__(WAVES * 64) adapter_few_kernel(AdapterKArgs a) {
  typedef Few<T, 1, NT, WAVES> F;
  constexpr int kSums = WAVES * NT * 1024;
  __shared__ __attribute__((aligned(1024))) char lds[kSums > WAVES * F::kLds ? kSums : WAVES * F::kLds];
  f32x4 (*sums)[NT][16][4] = reinterpret_cast<f32x4 (*)[NT][16][4]>(lds);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, i = lane & 15;
  const int c0 = blockIdx.x * 16, N = a.w.rows, R = a.rank;
  F few;
  const int steps = a.k / 64, left = a.k % 64;
  few.aim([&](int, int r) { return a.w.p + (int64_t)min(c0 + r, N - 1) * a.w.stride; },
          [&](int t, int r) { return a.x.p + (int64_t)min(t * 16 + r, a.x.rows - 1) * a.x.stride; }, 0, steps,
          blockIdx.x, lds + wave * F::kLds);
  few.prime(wave, WAVES);
  // The adapters' sums of this thread's results, while the first weights are on
  // their way: kRank of the rank at a time, whose low values, which 16 columns
  // share, are added up in LDS once.
  constexpr int kRank = 64, kThreads = WAVES * 64;
  constexpr int kMine = (NT * 256 + kThreads - 1) / kThreads;
  constexpr int kUnroll = WAVES > 8 ? 2 : 4;
  __shared__ __attribute__((aligned(16))) float lows[NT * 16][kRank + 4];
  float own[kMine] = {};
  int id[kMine];
#pragma unroll
  for (int m = 0; m < kMine; ++m) {
    const int o = m * kThreads + threadIdx.x, r = o >> 4;
    id[m] = r < a.x.rows && c0 + (o & 15) < N ? a.ids[r] : -1;
    if (id[m] >= a.adapters) id[m] = -1;
  }
  const int64_t plane = (int64_t)a.x.rows * a.low_stride;
  for (int k0 = 0; k0 < R; k0 += kRank) {
    if (k0) __syncthreads();
    for (int o = threadIdx.x; o < NT * kRank * 4; o += kThreads) {
      const int r = o / (kRank / 4), k = o % (kRank / 4) * 4;
      const float* low =
          static_cast<const float*>(a.low) + (int64_t)min(r, a.x.rows - 1) * a.low_stride + min(k0 + k, a.low_stride - 4);
      f32x4 v[kLowSplits];
#pragma unroll
      for (int s = 0; s < kLowSplits; ++s) v[s] = *reinterpret_cast<const f32x4*>(low + s * plane);
      f32x4 sum = v[0];
#pragma unroll
      for (int s = 1; s < kLowSplits; ++s) sum += v[s];
      *reinterpret_cast<f32x4*>(&lows[r][k]) = sum;
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < kMine; ++m) {
      if (id[m] < 0) continue;
      const int o = m * kThreads + threadIdx.x;
      const uint16_t* b = a.b + ((int64_t)id[m] * N + c0 + (o & 15)) * R;
#pragma unroll kUnroll
      for (int k = k0; k < min(k0 + kRank, R); k += 8) {
        u32x4 w[1];
        const uint32_t rows[1] = {0};
        b_elements<1>(b, rows, k, R, w);
        // (what is past the rank is 0 in both)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          own[m] += lows[o >> 4][k - k0 + e] * T::to_float((uint16_t)(w[0][e >> 1] >> (e & 1) * 16));
      }
    }
  }
  f32x4 acc[1][NT] = {};
  few.run(wave, WAVES, acc);
  if (left && steps % WAVES == wave) few.tail(left, acc);
  __syncthreads();                                        // the waves' pieces of lds become the sums
#pragma unroll
  for (int t = 0; t < NT; ++t) sums[wave][t][i][lane >> 4] = acc[0][t];
  __syncthreads();
  const float* sum = reinterpret_cast<const float*>(lds);
#pragma unroll
  for (int m = 0; m < kMine; ++m) {
    const int o = m * WAVES * 64 + threadIdx.x, r = o >> 4, c = c0 + (o & 15);
    if (r >= a.x.rows || c >= N) continue;
    float v = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) v += sum[(w * NT * 16 + r) * 16 + (o & 15)];
    v += own[m];
    const int64_t at = r * a.out_stride + c;
    if (a.out_f32) static_cast<float*>(a.out)[at] = v;
    else static_cast<uint16_t*>(a.out)[at] = T::from_float(v);
  }
}

// Adds the adapters' sums to a tile's results.
template <class G>
__device__ __forceinline__ void add_adapters(const AdapterKArgs& a, int pt, int qt, const int (&id)[G::FQ],
                                             typename G::Acc& acc) {
  typedef typename G::T T;
  const int lane = threadIdx.x & 63, quarter = lane >> 4;
  const int N = a.w.rows, R = a.rank;
  // Each of the waves that share k takes its part of the adapters; B of the
  // next one is loaded while this one's products are made.
  constexpr int kWaves = G::kThreads / 64, kGroups = G::kK / 64;
  static_assert(kWaves % kGroups == 0, "waves that share k");
  // Columns' fragments at a time, and whether the low values of all rows are
  // held at once, within the registers.  (float16 tiles of 256 x 256 still keep
  // 12 of them in scratch memory; with two fragments at a time none, but 4096
  // rows of 8192 x 1024 with 300 prompts take 152 us for 142.)
  constexpr bool kKeep = G::FP * G::FQ <= 16;
  constexpr int kPart = kKeep ? G::FP : 4;
  // Rows are found from the tile's first by 32-bit offsets (256 rows of 1024).
  uint32_t low[G::FQ];
  const uint16_t* low_base = static_cast<const uint16_t*>(a.low) + (int64_t)qt * G::TQ * a.low_stride;
#pragma unroll
  for (int j = 0; j < G::FQ; ++j) {
    const int q = G::wave_q() + j * 16 + (lane & 15), last = a.x.rows - 1 - qt * G::TQ;
    low[j] = (uint32_t)(min(q, last) * a.low_stride + quarter * 8) * 2;
  }
  const int64_t plane = (int64_t)a.x.rows * a.low_stride;
  uint64_t pending[G::FQ];
  // the next adapter that is left, or -1
  auto next = [&]() {
    int ad = -1;
#pragma unroll
    for (int j = 0; j < G::FQ; ++j)
      if (ad < 0 && pending[j]) ad = __builtin_amdgcn_readlane(id[j], __builtin_ctzll(pending[j]));
#pragma unroll
    for (int j = 0; j < G::FQ; ++j) pending[j] &= ~__ballot(id[j] == ad);
    return ad;
  };
  auto next_mine = [&]() {
    int mine = -1;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const int ad = next();
      if (g == G::wave_k()) mine = ad;
    }
    return mine;
  };
  for (int k = 0; k < R; k += 32) {
    auto load_low = [&](int j, u32x4 (&part)[kParts]) {
#pragma unroll
      for (int pl = 0; pl < kParts; ++pl)
        part[pl] = *reinterpret_cast<const u32x4*>(reinterpret_cast<const uint8_t*>(low_base + pl * plane + k) + low[j]);
    };
    auto load_b = [&](int ad, int i0, u32x4 (&b)[kPart]) {
      uint32_t rows[kPart];
#pragma unroll
      for (int i = 0; i < kPart; ++i)
        rows[i] = (uint32_t)(min(G::wave_p() + (i0 + i) * 16 + (lane & 15), N - 1 - pt * G::TP) * R) * 2;
      const uint16_t* base = a.b + ((int64_t)ad * N + pt * G::TP) * R;
      b_elements<kPart>(base, rows, k + quarter * 8, R, b);
    };
#pragma unroll
    for (int i0 = 0; i0 < G::FP; i0 += kPart) {
      u32x4 kept[kKeep ? G::FQ : 1][kParts];
#pragma unroll
      for (int j = 0; j < G::FQ; ++j) {
        if constexpr (kKeep) load_low(j, kept[j]);
        pending[j] = __ballot(id[j] >= 0 && id[j] < a.adapters);
      }
      int ad = next_mine();
      u32x4 b[kPart];
      if (ad >= 0) load_b(ad, i0, b);
      while (ad >= 0) {
        __builtin_amdgcn_sched_barrier(0);
        const int after = next_mine();
        u32x4 ahead[kPart];
        if (after >= 0) load_b(after, i0, ahead);
#pragma unroll
        for (int j = 0; j < G::FQ; ++j) {
          if (!__ballot(id[j] == ad)) continue;
          u32x4 part[kParts];
          if constexpr (kKeep) {
#pragma unroll
            for (int pl = 0; pl < kParts; ++pl) part[pl] = kept[j][pl];
          } else {
            load_low(j, part);
          }
          // float16: B's second part, which may be 0, and an infinite low value
          // do not meet.
          u32x4 finite = part[0];
          if constexpr (std::is_same<T, F16>::value) {
            if (__ballot(!all_finite(part[0]))) finite = finite_ones(part[0]);
          }
#pragma unroll
          for (int i = 0; i < kPart; ++i) {
            f32x4 sum = {0, 0, 0, 0};
            u32x4 v[2] = {b[i], {}};
            if constexpr (std::is_same<T, F16>::value) split_f16_finite(b[i], &v[0], &v[1]);
#pragma unroll
            for (int pl = 0; pl < kParts; ++pl) {
              sum = BF16::mfma(v[0], part[pl], sum);
              if constexpr (std::is_same<T, F16>::value) sum = BF16::mfma(v[1], pl ? part[pl] : finite, sum);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
              acc[i0 + i][j][e] = id[j] == ad ? acc[i0 + i][j][e] + sum[e] : acc[i0 + i][j][e];
          }
        }
        ad = after;
#pragma unroll
        for (int i = 0; i < kPart; ++i) b[i] = ahead[i];
      }
    }
  }
}

template <class G>
__global__ void __launch_bounds__(G::kThreads, G::kThreads / 256) adapter_kernel(AdapterKArgs a) {
  typedef typename G::T T;
  __shared__ __attribute__((aligned(1024))) char lds[G::kLds];
  int pt, qt;
  tile_of(a.ptiles, a.qtiles, &pt, &qt);
  typename G::SideP sp;
  typename G::SideQ sq;
  sp.aim(a.w, pt * G::TP);
  sq.aim(a.x, qt * G::TQ);
  G::begin((MOE_EP_LDS char*)lds, sp, sq, a.k);
  typename G::Acc acc;
  G::clear(acc);
  int id[G::FQ];                                          // of the wave's rows
#pragma unroll
  for (int j = 0; j < G::FQ; ++j) {
    const int q = qt * G::TQ + G::wave_q() + j * 16 + (threadIdx.x & 15);
    id[j] = q < a.x.rows ? a.ids[q] : -1;
  }
  G::loop((MOE_EP_LDS char*)lds, sp, sq, a.k, acc);
  add_adapters<G>(a, pt, qt, id, acc);
  if (!G::join((MOE_EP_LDS char*)lds, acc)) return;

  const int lane = threadIdx.x & 63, quarter = lane >> 4, N = a.w.rows;
#pragma unroll
  for (int j = 0; j < G::FQ; ++j) {
    const int q = qt * G::TQ + G::wave_q() + j * 16 + (lane & 15);
    if (q >= a.x.rows) continue;
#pragma unroll
    for (int i = 0; i < G::FP; ++i) {
      const int c = pt * G::TP + G::wave_p() + i * 16 + quarter * 4;
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = acc[i][j][e];
      store4<T>(a.out, q * a.out_stride + c, a.out_f32, N - c, v);
    }
  }
}

template <class G>
hipError_t adapter_tiles(AdapterKArgs a, hipStream_t stream) {
  a.ptiles = tiles(a.w.rows, G::TP);
  a.qtiles = tiles(a.x.rows, G::TQ);
  adapter_kernel<G><<<dim3(a.ptiles * a.qtiles), dim3(G::kThreads), 0, stream>>>(a);
  return hipGetLastError();
}
template <class T, int NT>
hipError_t adapter_few(const AdapterKArgs& a, hipStream_t stream) {
  const int blocks = tiles(a.w.rows, 16);
  if (NT > 2 || blocks >= 256) adapter_few_kernel<T, NT, 8><<<dim3(blocks), dim3(512), 0, stream>>>(a);
  else adapter_few_kernel<T, NT <= 2 ? NT : 2, 16><<<dim3(blocks), dim3(1024), 0, stream>>>(a);
  return hipGetLastError();
}
template <class T, int BLOCK, bool FEW>
hipError_t low(const AdapterKArgs& a, hipStream_t stream) {
  // 64 of the rank to a workgroup read x once for four times 16, where there
  // are workgroups enough all the same
  const int blocks = tiles(a.x.rows, BLOCK), parts = FEW ? kLowSplits : 1;
  if (a.rank > 32 && (int64_t)blocks * tiles(a.rank, 64) * parts >= 128)
    low_kernel<T, BLOCK, 4, FEW><<<dim3(blocks, tiles(a.rank, 64), parts), dim3(kLowWaves * 64), 0, stream>>>(a);
  else
    low_kernel<T, BLOCK, 1, FEW><<<dim3(blocks, tiles(a.rank, 16), parts), dim3(kLowWaves * 64), 0, stream>>>(a);
  return hipGetLastError();
}
template <class T>
hipError_t adapter(const AdapterKArgs& a, hipStream_t stream) {
  static_assert(kLowFew == 64, "the few kernels' rows");
  const int n = a.x.rows;
  const hipError_t e = n <= kLowFew      ? low<T, 1, true>(a, stream)
                       : n <= kLowSingle ? low<T, 1, false>(a, stream)
                                         : low<T, 8, false>(a, stream);
  if (e != hipSuccess) return e;
  if (n <= 16) return adapter_few<T, 1>(a, stream);
  if (n <= 32) return adapter_few<T, 2>(a, stream);
  if (n <= 48) return adapter_few<T, 3>(a, stream);
  if (n <= 64) return adapter_few<T, 4>(a, stream);
  const bool direct = a.w.whole && a.x.whole;
  switch (tile_size(a.w.rows, a.x.rows, a.k, direct, true)) {
    case k256x256: return adapter_tiles<Gemm<T, true, true, false, 256, 256, 2, 4, 1, true>>(a, stream);
    case k256x128: return adapter_tiles<Gemm<T, true, true, false, 256, 128, 2, 4, 1, true>>(a, stream);
    case k128x128:
      return direct ? adapter_tiles<Gemm<T, true, true, false, 128, 128, 2, 2, 2, true>>(a, stream)
                    : adapter_tiles<Gemm<T, true, true, false, 128, 128, 2, 2, 2, false>>(a, stream);
    case k64x64:
      return direct ? adapter_tiles<Gemm<T, true, true, false, 64, 64, 2, 2, 4, true>>(a, stream)
                    : adapter_tiles<Gemm<T, true, true, false, 64, 64, 2, 2, 4, false>>(a, stream);
    default:
      return direct ? adapter_tiles<Gemm<T, true, true, false, 32, 32, 1, 1, 4, true>>(a, stream)
                    : adapter_tiles<Gemm<T, true, true, false, 32, 32, 1, 1, 4, false>>(a, stream);
  }
}

}  // namespace

hipError_t launch_adapter(const AdapterKArgs& a, int dtype, hipStream_t stream) {
  return dtype == MOE_EP_BF16 ? adapter<BF16>(a, stream) : adapter<F16>(a, stream);
}

}  // namespace moe_ep_detail
