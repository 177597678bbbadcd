// Attention over the paged NVFP4 key/value cache.
//
// For a query row q at position i and the keys and values of its request:
//   s_j = scale * d_k * (q . K_j),  p_j = exp(s_j - m),  out = d_v * sum_j p_j V_j / sum_j p_j,
//   lse = m + ln sum_j p_j, over the positions j <= i (and j > i - window).
// K_j and V_j are e2m1 * e4m3, built in registers as fp16 matrix operands (exact); a query row enters as
// fp16 after scaling by a power of two that puts its largest element in [2^14, 2^15) (exact for every
// element within 2^-31 of it), undone in the fp32 scores.  Scores, maxima, sums and outputs are fp32;
// p_j is rounded to fp16 (11 bits, 8 times finer than the bf16 output) for the value product.
//
// Both products keep the cache operand first: S^T = K Q^T leaves, in each lane, the scores of one query
// row, and the eight (sixteen) keys a lane then holds are the contraction elements of its operand in
// O^T = V^T P^T when the keys are taken in that order, which is the order the value codes are stored
// in: p goes from one product into the next without leaving its lane.
//
// The running maximum is a reference that only moves when a score exceeds it by more than 2^8 (in
// powers of two): p_j <= 2^8 relative to it, so the sums stay in range and exact in the same way, and
// the usual unit needs no exchange between lanes and no rescale.  p carries another factor 2^7, which
// cancels in out, so that fp16 p reaches down to 2^-31 of the largest.
//
// Exponents are fma(s, c, 7 - m), s the raw score of the product, c its factor and m = fl(max s * c): they differ
// from those relative to the exact maximum by the rounding of m, one number for the whole row, which cancels in
// out.  It must not reach a power of two, let alone the range of fp16: from |m| = 2^16 on (rounding 2^-8) a row is
// "far", its m is held as a raw score and its exponents are fma(s - m, c, 7), exactly 7 at the largest score.
#include "kv_launch.h"
#include "kv_operands.h"
#include "kv_schedule.h"

namespace moe {
namespace {

struct KvPartials {
  float* o;    // [slot][BM][D], unnormalised
  float* ml;   // [slot][2][BM]: reference maximum, sum
};

// ------------------------------------------------------------------------- few rows per request
// Workgroups of NW waves (4; 8 where whole tiles are taken) with an equal share of the units each (KvShare);
// of a segment (one kv head and row tile of 16*MI rows) each wave takes every NW-th unit.  A unit's 36*D
// contiguous bytes go straight to LDS, into a ring of kRing units of the wave's own (no barrier, no registers
// held for loads in flight), and from there to registers when their turn comes.  The waves' sums meet in LDS
// at the end of the segment.  MI = 2 where a request may have more than 16 rows per kv head.
// Bound by memory and the vector unit together: a unit of dimension 128 takes about 300 vector instructions of
// a wave, 1200 cycles, in which a quarter of a compute unit's share of the memory brings 4.6 KB.  64 requests
// of 90 to 8100 positions (64/8 heads, 313 MB): 62 us and 7 us for the combine launch, 4.5 TB/s over both; 3
// contexts of 70 to 131 thousand positions (32/8 heads, 372 MB): 5.0 TB/s; a plain read reaches 7.1 TB/s.
template <int D, int MI, int NW>
__global__ __launch_bounds__(64 * NW, (rows_occupancy<D, MI, NW>())) void kv_attention_rows_kernel(
    KvAttentionProblem a, KvSchedule s, KvPartials part) {
  using U = KvUnit<D>;
  constexpr int NS = D / 32, BM = 16 * MI, NL = NS / 2;
  constexpr int kFull = U::kBytes / 1024, kTail = U::kBytes % 1024 / 256;   // 1024- and 256-byte loads of a unit
  constexpr int kOut = NW * BM * 36 * 4, kRings = NW * kRing * U::kBytes;
  // the waves' rings; at the end of a segment one 32-element range of the sums (rows padded to 36 floats)
  __shared__ __align__(16) uint8_t lds[kOut > kRings ? kOut : kRings];
  __shared__ float m_lds[NW][BM], l_lds[NW][BM];
  if (blockIdx.x >= a.work_groups) return kv_fill_rows<D>(a, blockIdx.x - a.work_groups, gridDim.x - a.work_groups);
  using lds_bytes = __attribute__((address_space(3))) uint8_t*;
  float(*o_lds)[BM][36] = reinterpret_cast<float(*)[BM][36]>(lds);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int q4 = lane >> 4, n16 = lane & 15;
  const int hkv = a.cache.kv_heads;
  const lds_bytes ring = (lds_bytes)lds + wave * kRing * U::kBytes;
  KvShare sh;
  KvWhere at;
  long long local;
  constexpr bool kWhole = NW > 4;     // a whole tile per workgroup
  if (!kv_locate<kWhole>(a, s, blockIdx.x, &sh, &at, &local)) return;
  int left = kWhole ? max(1, at.q.units) : (int)min(sh.chunk, sh.total - (long long)blockIdx.x * sh.chunk);
  const int chunk = (int)min(sh.chunk, (long long)(1 << 28));
  const int upp = a.cache.page_size / kKvUnit;
  bool first = true;

  while (true) {
    const int units = max(1, at.q.units);
    const long long step = kWhole ? 1 : kv_step(at.q, sh), nth = div_i64(local, step);
    // place in the tile: `lead` empty places before unit 0
    const int lead = kWhole || sh.aligned ? 0 : kSwitch, place = (int)(local - nth * step), unit = max(0, place - lead);
    const int h = (int)div_i64(nth, at.q.tiles), tile = (int)(nth - (long long)h * at.q.tiles);
    const int taken = min(left, lead + units - place), count = place + taken - lead - unit;
    if (count <= 0) return;       // the share ends before the tile's first unit

    const int rows = at.q.n * a.G, row_base = tile * BM;
    const int pos0 = at.q.len - at.q.n;          // position of the request's first row
    // positions seen by the tile's rows: every row sees [see_all, pos_min], none anything before see_any
    const int pos_min = pos0 + row_base / a.G, pos_max = pos0 + (min(row_base + BM, rows) - 1) / a.G;
    const int see_all = a.window > 0 ? (int)max(0ll, (long long)pos_max - a.window + 1) : 0;
    const int see_any = a.window > 0 ? (int)max(0ll, (long long)pos_min - a.window + 1) : 0;
    const int u0 = see_any / kKvUnit + unit;
    const int u1 = pos_max < 0 ? u0 : min(u0 + count, pos_max / kKvUnit + 1);
    const int32_t* table = a.table + (size_t)at.r * a.width;

    // the wave's units u0 + wave + NW*i, i < mine; lane i & 63 holds the address of unit i of a batch of 64
    // (0 for a bad table entry), bad[batch & 1] the bad ones
    const int ufirst = u0 + wave, mine = ufirst < u1 ? (u1 - ufirst + NW - 1) / NW : 0;
    uint64_t where = 0, bad[2] = {0, 0};
    auto issue = [&](int i, int slot) {
      if ((i & 63) == 0) {
        const int uu = ufirst + NW * (i + lane);
        where = 0;
        if (i + lane < mine) {
          const int b = uu / upp, p = b < a.width ? table[b] : -1;
          if (p >= 0 && p < a.cache.num_pages)
            where = reinterpret_cast<uint64_t>(a.cache.pages) +
                    (((uint64_t)p * hkv + h) * upp + (uu - b * upp)) * (uint64_t)U::kBytes;
        }
        const uint64_t none = __ballot(where == 0);
        if (i & 64) bad[1] = none;
        else bad[0] = none;
      }
      const uint64_t at_unit = (uint64_t)lane_i64((long long)where, i & 63);
      const uint8_t* base = at_unit ? reinterpret_cast<const uint8_t*>(at_unit) : a.cache.pages;
      const uint32_t dst = (uint32_t)(uintptr_t)ring + slot * U::kBytes;
#pragma unroll
      for (int j = 0; j < kFull; ++j) direct_load16_nt(base + 1024 * j, 16 * lane, dst + 1024 * j);
#pragma unroll
      for (int j = 0; j < kTail; ++j)
        direct_load4_nt(base + 1024 * kFull + 256 * j, 4 * lane, dst + 1024 * kFull + 256 * j);
    };
    if (!first) __syncthreads();      // the previous segment's reads of LDS
    for (int i = 0; i < min(mine, kRing); ++i) issue(i, i);

    // query operands: row n16 of block mi, elements [32s + 8*q4, +8)
    f16x8 qf[MI][NS];
    float c[MI];
    int pos[MI];
#pragma unroll
    for (int mi = 0; mi < MI; ++mi) {
      const int row = row_base + 16 * mi + n16;
      const bool valid = row < rows;
      const int tok = valid ? row / a.G : 0, g = valid ? row - tok * a.G : 0;
      pos[mi] = valid ? pos0 + tok : -1;
      const uint16_t* src = a.q + (int64_t)(at.q.row0 + tok) * a.q_stride + (size_t)(h * a.G + g) * D + 8 * q4;
      u32x4 w[NS];
      uint32_t top = 0;
#pragma unroll
      for (int k = 0; k < NS; ++k) {
        w[k] = *reinterpret_cast<const u32x4*>(src + 32 * k);
#pragma unroll
        for (int j = 0; j < 4; ++j) top = max(top, max(w[k][j] & 0x7FFFu, (w[k][j] >> 16) & 0x7FFFu));
      }
      int e = (int)(top >> 7);    // the row's largest exponent field
      e = max(e, __shfl_xor(e, 16));
      e = max(e, __shfl_xor(e, 32));
      const int shift = row_shift(e, a.scale * kLog2e);
#pragma unroll
      for (int k = 0; k < NS; ++k) {
        const f16x2 p0 = bf16x2_to_f16(w[k][0], shift), p1 = bf16x2_to_f16(w[k][1], shift);
        const f16x2 p2 = bf16x2_to_f16(w[k][2], shift), p3 = bf16x2_to_f16(w[k][3], shift);
        qf[mi][k] = f16x8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
      }
      c[mi] = fminf(ldexpf(a.scale * kLog2e, -shift), FLT_MAX);      // a score of 0 stays 0
    }

    f32x4 o[MI][NS][2];
    float m[MI], l[MI];
    bool far[MI], any_far = false;
#pragma unroll
    for (int mi = 0; mi < MI; ++mi) {
      far[mi] = false;
      m[mi] = kNone;
      l[mi] = 0.f;
#pragma unroll
      for (int r = 0; r < NS; ++r) o[mi][r][0] = o[mi][r][1] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    // `off`: byte of the ring where the unit begins
    auto compute = [&](int uu, int off, bool bad_page) {
      const int key0 = kKvUnit * uu;
      const lds_bytes unit_lds = ring + off;
      u32x4 kc[NL];
      uint32_t ks[NS / 2];      // 2*NS scale bytes: word w = block*NS + step
#pragma unroll
      for (int j = 0; j < NL; ++j)
        kc[j] = *reinterpret_cast<const __attribute__((address_space(3))) u32x4*>(unit_lds + 1024 * j + 16 * lane);
#pragma unroll
      for (int j = 0; j < NS / 2; ++j)
        ks[j] = *reinterpret_cast<const __attribute__((address_space(3))) uint32_t*>(
            unit_lds + U::kKScales + (16 * (q4 >> 1) + n16) * 2 * NS + 4 * j);
      f32x4 sc[MI][2];
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
#pragma unroll
        for (int mi = 0; mi < MI; ++mi) sc[mi][kb] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < NS; ++k) {
          const int w = kb * NS + k;
          const f16x2 sp = scale_pair(ks[w >> 2], (w & 2) != 0);
          const f16x8 kf = k_operand(kc[w >> 2][w & 3], (w & 1) ? sp[1] : sp[0]);
#pragma unroll
          for (int mi = 0; mi < MI; ++mi)
            sc[mi][kb] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, qf[mi][k], sc[mi][kb], 0, 0, 0);
        }
      }
      // units that some row does not see whole: masks, and nothing from positions past the length
      const bool whole = key0 + kKvUnit - 1 <= pos_min && key0 >= see_all;
      if (!whole || bad_page) {
        const int quarter = 4 * (lane_now() >> 4);
#pragma unroll
        for (int mi = 0; mi < MI; ++mi)
#pragma unroll
          for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int key = key0 + 16 * kb + quarter + k;
              const bool seen = key <= pos[mi] && (a.window == 0 || pos[mi] - key < a.window);
              sc[mi][kb][k] = !seen ? -INFINITY : bad_page ? NAN : sc[mi][kb][k];
            }
        // value scales of positions past the length to zero, in the ring
        const u32x2 keep = {bad_page ? 0u : keep_bytes(key0 + quarter, at.q.len),
                            bad_page ? 0u : keep_bytes(key0 + 16 + quarter, at.q.len)};
        const int half = (lane_now() & 15) >> 3;
#pragma unroll
        for (int r = 0; r < NS; ++r) {
          auto* vs = reinterpret_cast<__attribute__((address_space(3))) u32x2*>(
              unit_lds + U::kVScales + ((quarter / 2 + half) * NS + r) * 8);
          *vs &= keep;      // the eight lanes that share the bytes write the same
        }
      }
      f16x8 pf[MI];
#pragma unroll
      for (int mi = 0; mi < MI; ++mi) {
        float t[8];
        auto exponents = [&]() {
          const float ref = m[mi] - kPExp;
#pragma unroll
          for (int k = 0; k < 8; ++k) t[k] = __fmaf_rn(sc[mi][k >> 2][k & 3], c[mi], -ref);
          if (__builtin_expect(any_far, 0)) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              t[k] = far[mi] ? __fmaf_rn(sc[mi][k >> 2][k & 3] - m[mi], c[mi], kPExp) : t[k];
          }
        };
        exponents();
        const float most =
            fmaxf(fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])), fmaxf(fmaxf(t[4], t[5]), fmaxf(t[6], t[7])));
        if (__any(most > kSlack + kPExp)) {
          float mx = -INFINITY;
#pragma unroll
          for (int k = 0; k < 8; ++k) mx = fmaxf(mx, sc[mi][k >> 2][k & 3]);
          const float f = kv_move(quarter_max(mx), c[mi], m[mi], far[mi]);
          any_far |= __any(far[mi]);
          l[mi] *= f;
#pragma unroll
          for (int r = 0; r < NS; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int k = 0; k < 4; ++k) o[mi][r][e][k] *= f;
          exponents();
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) t[k] = exp2_hw(t[k]);
        l[mi] += ((t[0] + t[1]) + (t[2] + t[3])) + ((t[4] + t[5]) + (t[6] + t[7]));
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const f16x2 pr = __builtin_convertvector((f32x2){t[k], t[4 + k]}, f16x2);      // the order of v_octet
          pf[mi][2 * k] = pr[0];
          pf[mi][2 * k + 1] = pr[1];
        }
      }
#pragma unroll
      for (int r = 0; r < NS; ++r) {
        const u32x2 vc = *reinterpret_cast<const __attribute__((address_space(3))) u32x2*>(
            unit_lds + U::kVCodes + 1024 * (r >> 1) + 16 * lane + 8 * (r & 1));
        const u32x2 vs = *reinterpret_cast<const __attribute__((address_space(3))) u32x2*>(
            unit_lds + U::kVScales + ((2 * q4 + (n16 >> 3)) * NS + r) * 8);
        f16x8 ve, vo;
        v_octet(vc[0], vc[1], vs[0], vs[1], &ve, &vo);
#pragma unroll
        for (int mi = 0; mi < MI; ++mi) {
          o[mi][r][0] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ve, pf[mi], o[mi][r][0], 0, 0, 0);
          o[mi][r][1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vo, pf[mi], o[mi][r][1], 0, 0, 0);
        }
      }
    };

    for (int i = 0, slot = 0; i < mine; ++i) {
      // Waves that have most of their share left go first: the scheduler prefers the oldest wave, which
      // finishes its share while the youngest has the compute unit to itself at the end, too few to hide
      // latency (shares of equal length took 22 to 72 us).
      const int rest = left - NW * i;
      if (4 * rest > 3 * chunk) __builtin_amdgcn_s_setprio(3);
      else if (2 * rest > chunk) __builtin_amdgcn_s_setprio(2);
      else if (4 * rest > chunk) __builtin_amdgcn_s_setprio(1);
      else __builtin_amdgcn_s_setprio(0);
      wait_units<kFull + kTail>(min(kRing, mine - i) - 1);
      compute(ufirst + NW * i, slot * U::kBytes, (bad[(i >> 6) & 1] >> (i & 63)) & 1);
      if (i + kRing < mine) {
        asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");   // the slot has been read
        issue(i + kRing, slot);
      }
      slot = slot + 1 == kRing ? 0 : slot + 1;
    }

    // the waves' sums: common reference maximum per row, then range by range through LDS
    __syncthreads();      // every wave has read its ring
    const int elane = lane_now(), eq = elane >> 4, en = elane & 15, etid = 64 * wave + elane;
#pragma unroll
    for (int mi = 0; mi < MI; ++mi) {
      const float ls = quarter_sum(l[mi]);
      m[mi] = kv_reference(m[mi], c[mi], far[mi]);
      if (eq == 0) {
        m_lds[wave][16 * mi + en] = m[mi];
        l_lds[wave][16 * mi + en] = ls;
      }
    }
    __syncthreads();
    float f[MI];
#pragma unroll
    for (int mi = 0; mi < MI; ++mi) {
      const int rr = 16 * mi + en;
      float top = m_lds[0][rr];
#pragma unroll
      for (int w = 1; w < NW; ++w) top = fmaxf(top, m_lds[w][rr]);
      f[mi] = exp2_hw(m[mi] - top);
    }
    const bool direct = count == units;
    // of the first 256 threads: thread -> row tid / (256 / BM), consecutive elements of the range
    constexpr int TPR = 256 / BM, EPT = 32 / TPR;
    const int orow = (etid & 255) / TPR, oc = (etid % TPR) * EPT;
    float top = kNone, sum = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) top = fmaxf(top, m_lds[w][orow]);
#pragma unroll
    for (int w = 0; w < NW; ++w) sum += l_lds[w][orow] * exp2_hw(m_lds[w][orow] - top);
    const int grow = row_base + orow;
    const bool valid = grow < rows && etid < 256;
    const int tok = grow / a.G, g = grow - tok * a.G;
    const size_t dst_row = (size_t)(at.q.row0 + tok) * a.Hq + h * a.G + g;
    const size_t slot = 2 * (size_t)blockIdx.x + (unit == 0 ? 1 : 0);
    const float norm = sum > 0.f || sum != sum ? a.cache.v_gscale / sum : 0.f;
    if (etid % TPR == 0 && valid) {
      if (direct) {
        if (a.lse)
          a.lse[dst_row] = sum > 0.f || sum != sum ? kLn2 * (top + (__builtin_amdgcn_logf(sum) - kPExp)) : -INFINITY;
      } else {
        part.ml[slot * 2 * BM + orow] = top;
        part.ml[slot * 2 * BM + BM + orow] = sum;
      }
    }
#pragma unroll
    for (int r = 0; r < NS; ++r) {
      if (r > 0) __syncthreads();
#pragma unroll
      for (int mi = 0; mi < MI; ++mi) {
        float* dst = &o_lds[wave][16 * mi + en][8 * eq];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          dst[2 * k] = o[mi][r][0][k] * f[mi];
          dst[2 * k + 1] = o[mi][r][1][k] * f[mi];
        }
      }
      __syncthreads();
      float v[EPT];
#pragma unroll
      for (int e = 0; e < EPT; ++e)
        v[e] = 0.f;
#pragma unroll
      for (int w = 0; w < NW; w += 2)
#pragma unroll
        for (int e = 0; e < EPT; ++e) v[e] += o_lds[w][orow][oc + e] + o_lds[w + 1][orow][oc + e];
      if (valid) {
        if (direct) {
          uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + dst_row * D + 32 * r + oc);
#pragma unroll
          for (int e = 0; e < EPT / 2; ++e) dst[e] = f32x2_to_bf16x2(v[2 * e] * norm, v[2 * e + 1] * norm);
        } else {
          float* dst = part.o + (slot * BM + orow) * D + 32 * r + oc;
#pragma unroll
          for (int e = 0; e < EPT; ++e) dst[e] = v[e];
        }
      }
    }

    // the next segment: of this request, or of the next one with rows
    left -= taken;
    if (kWhole || left == 0 || sh.aligned) return;
    first = false;
    local += taken;
    if (local == kv_units(at.q, sh) * hkv) {
      local = 0;
      do {
        at.q = lane_request(kv_request(a, s, ++at.r), 0);      // the share ends within the last request
      } while (at.q.tiles == 0);
    }
  }
}

// ------------------------------------------------------------------------ many rows per request
// One workgroup (NW waves of RS rows) per (kv head, row tile, split).  NU units (32 positions each) at a
// time are dequantized once into LDS, as fp16 operands in fragment order (lane l's 16 bytes at 16*l), and
// multiplied by every wave; the next step's codes are in registers and its operands written to the other
// LDS buffer meanwhile.
// RS = 32, the 32x32x16 instruction:
//   key operand, unit b, step t (16 elements): lane 32z + p holds position p, elements [16t + 8z, +8)
//   value operand, unit b, step t (16 positions), range r: lane 32z + d holds element 32r + d, positions
//     16t + 4z + {0..3} and 16t + 8 + 4z + {0..3}: the ones whose scores lane 32z + n holds after S^T.
// RS = 16, the 16x16x32 instruction: the operands as the cache holds them (value operand, range r: the
//   even elements, then the odd ones).  Half the rows per operand read, which LDS bandwidth then bounds at
//   half the matrix rate, and twice the tiles.  Taken where those fill the card better (plan_launches), and
//   for head dimension 256, whose 32-row outputs and queries (128 + 64 of 256 registers) leave none to
//   overlap anything: 175 us against 350 us for the chunks of 5 requests (16/2 heads, window 1024).
// Bound by the vector unit and LDS beside the matrix unit: a prompt of 8192 (32/8 heads, dimension 128)
// runs at 975-1002 TFLOP/s, the matrix unit 46% busy, 7.0 vector instructions beside each 32-cycle matrix
// instruction (32 exponentials, 32 fused multiply-adds, 37 additions, 16 conversions, 16 maxima and the
// wave's eighth of the dequantization per 32 of them).  The chunks (dimension 256) run at 470 TFLOP/s, the matrix unit
// 25% busy, 5.2 vector instructions beside each 16-cycle one: matrix, LDS and vector work of a step of one unit follow
// one another, with two waves per SIMD in step and a barrier every 32 positions, and about 620 items make 2.4 rounds of
// the 256 places.
template <int D, int NW, int NU, int RS>
__global__ __launch_bounds__(64 * NW, 2) void kv_attention_tiles_kernel(KvAttentionProblem a, KvSchedule s,
                                                                        KvPartials part) {
  using U = KvUnit<D>;
  constexpr int NS = D / 32, NT = D / 16, BM = RS * NW, THREADS = 64 * NW;
  constexpr bool kWide = RS == 32;
  constexpr int NQ = kWide ? NT : NS;                 // query operands
  constexpr int NSC = kWide ? 16 : 8;                 // scores of a lane and unit
  constexpr int kHalf = 2 * D * NU;                   // 8-byte code pieces of the keys (and of the values) of a step
  constexpr int kKeys = 64 * D * NU;                  // bytes of the keys' (and of the values') operands
  __shared__ __align__(16) uint8_t key_lds0[kKeys], key_lds1[kKeys], value_lds0[kKeys], value_lds1[kKeys];
  if (blockIdx.x >= a.work_groups) return kv_fill_rows<D>(a, blockIdx.x - a.work_groups, gridDim.x - a.work_groups);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int z = lane / RS, nrow = lane & (RS - 1);     // part of the contraction, row
  const int hkv = a.cache.kv_heads;
  const int h = blockIdx.x % hkv;
  KvItem it;
  if (!kv_find<false>(a, s, blockIdx.x / hkv, &it)) return;
  {
    // late rows see the most: their tiles first
    const int t = it.q.tiles - 1 - it.tile;
    it.slot += (t - it.tile) * it.splits;
    it.tile = t;
  }
  const int rows = it.q.n * a.G, row_base = it.tile * BM;
  const int pos0 = it.q.len - it.q.n;

  // positions that the rows of [first, last) see: all of [*see_all, *pos_min], none outside
  // [*see_any, *pos_max]
  auto reach = [&](int first, int last, int* pos_min, int* pos_max, int* see_all, int* see_any) {
    *pos_min = pos0 + first / a.G;
    *pos_max = pos0 + (min(last, rows) - 1) / a.G;
    *see_all = a.window > 0 ? (int)max(0ll, (long long)*pos_max - a.window + 1) : 0;
    *see_any = a.window > 0 ? (int)max(0ll, (long long)*pos_min - a.window + 1) : 0;
  };
  int pos_min, pos_max, see_all, see_any, u0, u1;
  {
    int t0, t1, t2, t3;
    reach(row_base, row_base + BM, &t0, &t1, &t2, &t3);
    u0 = t3 / kKvUnit + it.split * it.chunk;
    u1 = t1 < 0 ? u0 : min(u0 + min(it.chunk, it.q.units - it.split * it.chunk), t1 / kKvUnit + 1);
  }
  if (u0 >= u1 && it.splits > 1) {      // nothing in this split: an empty partial sum, whose outputs are not read
    const size_t slot = (size_t)(it.slot + it.split) * hkv + h;
    for (int r = tid; r < min(BM, rows - row_base); r += THREADS) {
      part.ml[slot * 2 * BM + r] = kNone;
      part.ml[slot * 2 * BM + BM + r] = 0.f;
    }
    return;
  }

  // query operands: row nrow of the wave, elements [16t + 8z, +8) (RS = 16: [32t + 8z, +8))
  const int row = row_base + RS * wave + nrow;
  const bool valid = row < rows;
  const int tok = valid ? row / a.G : 0, g = valid ? row - tok * a.G : 0;
  int pos = valid ? pos0 + tok : -1;
  f16x8 qf[NQ];
  float c;
  {
    const uint16_t* src = a.q + (int64_t)(it.q.row0 + tok) * a.q_stride + (size_t)(h * a.G + g) * D + 8 * z;
    u32x4 w[NQ];
    uint32_t top = 0;
#pragma unroll
    for (int t = 0; t < NQ; ++t) {
      w[t] = *reinterpret_cast<const u32x4*>(src + (kWide ? 16 : 32) * t);
#pragma unroll
      for (int j = 0; j < 4; ++j) top = max(top, max(w[t][j] & 0x7FFFu, (w[t][j] >> 16) & 0x7FFFu));
    }
    int e = (int)(top >> 7);
    e = max(e, __shfl_xor(e, 32));
    if (!kWide) e = max(e, __shfl_xor(e, 16));
    const int sh = row_shift(e, a.scale * kLog2e);
#pragma unroll
    for (int t = 0; t < NQ; ++t) {
      const f16x2 p0 = bf16x2_to_f16(w[t][0], sh), p1 = bf16x2_to_f16(w[t][1], sh);
      const f16x2 p2 = bf16x2_to_f16(w[t][2], sh), p3 = bf16x2_to_f16(w[t][3], sh);
      qf[t] = f16x8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
    }
    c = fminf(ldexpf(a.scale * kLog2e, -sh), FLT_MAX);      // a score of 0 stays 0
  }
  const int wrow = row_base + RS * wave;
  reach(min(wrow, rows - 1), wrow + RS, &pos_min, &pos_max, &see_all, &see_any);
  // the last step may reach into the unit behind this split: nothing from `end` on counts
  const int end = min(it.q.len, (int)min((long long)u1 * kKvUnit, 0x7FFFFFFFll));
  const int low = a.window > 0 ? (int)max(0ll, (long long)pos - a.window + 1) : 0;
  pos = min(pos, end - 1);
  pos_min = min(pos_min, end - 1);

  // RS = 32: element 32r + 8(i/4) + 4z + i%4 in o[r][i]; RS = 16: 32r + 8z + 2i + e in o[2r + e][i]
  using Acc = std::conditional_t<kWide, f32x16, f32x4>;
  constexpr int NO = kWide ? NS : 2 * NS, NA = kWide ? 16 : 4;
  Acc o[NO];
  float m = kNone, l = 0.f;
  bool far = false, any_far = false;
#pragma unroll
  for (int r = 0; r < NO; ++r)
#pragma unroll
    for (int i = 0; i < NA; ++i) o[r][i] = 0.f;

  const int upp = a.cache.page_size / kKvUnit;
  const int32_t* table = a.table + (size_t)it.r * a.width;
  // addresses of a step's units (any valid unit past the end or for a bad table entry) and the bad ones' bits
  struct Step {
    uint64_t at[NU];
    uint32_t none;
  };
  uint64_t where = 0;      // lane i: address of unit u0 + 64*batch + i, 0 for a bad table entry
  auto locate = [&](int u) __attribute__((always_inline)) {
    if (((u - u0) & 63) == 0) {
      const int uu = u + lane, b = uu / upp;
      where = reinterpret_cast<uint64_t>(a.cache.pages);
      if (uu < u1) {
        const int p = b < a.width ? table[b] : -1;
        where = p >= 0 && p < a.cache.num_pages ? where + (((uint64_t)p * hkv + h) * upp + (uu - b * upp)) * (uint64_t)U::kBytes
                                                : 0;
      }
    }
    Step x;
    x.none = 0;
#pragma unroll
    for (int b = 0; b < NU; ++b) {
      x.at[b] = (uint64_t)lane_i64((long long)where, (u + b - u0) & 63);
      x.none |= x.at[b] == 0 ? 1u << b : 0u;
      if (x.at[b] == 0) x.at[b] = reinterpret_cast<uint64_t>(a.cache.pages);
    }
    return x;
  };
  // 8-byte code pieces of the keys (values) of a step: piece p = tid + THREADS*j, of unit b = p / 2D the piece
  // x = p % 2D: lane (x / 2) % 64 of the 16-row operand, words 2*(x%2).. of its 16-byte load x / 128
  // (a wave's pieces are all of one unit)
  constexpr int kPieces = (kHalf + THREADS - 1) / THREADS;
  u32x2 kcode[kPieces], vcode[kPieces], vscale[kPieces];
  uint32_t kscale[kPieces];
  auto first_piece = [&](int j) { return 64 * wave + THREADS * j; };
  auto beyond = [&](int j) { return kHalf < THREADS && first_piece(j) >= kHalf; };      // fewer pieces than threads
  auto load_keys = [&](const Step& st) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      if (beyond(j)) continue;
      const int b = first_piece(j) / (2 * D), x = (first_piece(j) & (2 * D - 1)) + lane;
      const uint8_t* ub = reinterpret_cast<const uint8_t*>(b ? st.at[NU - 1] : st.at[0]);
      const int ln = (x >> 1) & 63, w = 4 * (x >> 7) + 2 * (x & 1);
      kcode[j] = *reinterpret_cast<const u32x2*>(ub + 8 * x);
      kscale[j] = *reinterpret_cast<const uint16_t*>(ub + U::kKScales + (16 * (ln >> 5) + (ln & 15)) * 2 * NS + w);
    }
  };
  auto load_values = [&](const Step& st) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      if (beyond(j)) continue;
      const int b = first_piece(j) / (2 * D), x = (first_piece(j) & (2 * D - 1)) + lane;
      const uint8_t* ub = reinterpret_cast<const uint8_t*>(b ? st.at[NU - 1] : st.at[0]);
      const int ln = (x >> 1) & 63, r = 2 * (x >> 7) + (x & 1);
      vcode[j] = *reinterpret_cast<const u32x2*>(ub + U::kVCodes + 8 * x);
      vscale[j] = *reinterpret_cast<const u32x2*>(ub + U::kVScales +
                                                  ((2 * (ln >> 4) + ((ln & 15) >> 3)) * NS + r) * 8);
    }
  };
  auto store_keys = [&](uint8_t* dst) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      if (beyond(j)) continue;
      const int b = first_piece(j) / (2 * D), x = (first_piece(j) & (2 * D - 1)) + lane;
      const int ln = (x >> 1) & 63, w = 4 * (x >> 7) + 2 * (x & 1), q4 = ln >> 4, n16 = ln & 15;
      const f16x2 sp = scale_pair(kscale[j], false);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int kb = (w + e) / NS, i = (w + e) % NS;
        uint8_t* d = kWide ? dst + (b * NT + 2 * i + (q4 >> 1)) * 1024 + 16 * (32 * (q4 & 1) + 16 * kb + n16)
                           : dst + (b * NT + w + e) * 1024 + 16 * ln;
        *reinterpret_cast<f16x8*>(d) = k_operand(kcode[j][e], sp[e]);
      }
    }
  };
  auto store_values = [&](int u, const Step& st, uint8_t* dst) __attribute__((always_inline)) {
    if (__builtin_expect(kKvUnit * (u + NU) > end || st.none != 0, 0)) {
      // nothing from positions past the end or of bad pages
      asm volatile("");      // keeps this a branch
#pragma unroll
      for (int j = 0; j < kPieces; ++j) {
        if (beyond(j)) continue;
        const int b = first_piece(j) / (2 * D), x = (first_piece(j) & (2 * D - 1)) + lane;
        const int key0 = kKvUnit * (u + b) + 4 * ((x >> 5) & 3);
        vscale[j][0] &= (st.none >> b) & 1u ? 0u : keep_bytes(key0, end);
        vscale[j][1] &= (st.none >> b) & 1u ? 0u : keep_bytes(key0 + 16, end);
      }
    }
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      if (beyond(j)) continue;
      const int b = first_piece(j) / (2 * D), x = (first_piece(j) & (2 * D - 1)) + lane;
      const int ln = (x >> 1) & 63, r = 2 * (x >> 7) + (x & 1), q4 = ln >> 4, n16 = ln & 15;
      f16x4 even[2], odd[2];
      v_quad(vcode[j][0], vscale[j][0], &even[0], &odd[0]);
      v_quad(vcode[j][1], vscale[j][1], &even[1], &odd[1]);
      if (kWide) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          // positions 4*q4..: lane half z = q4 & 1, bytes 8*(q4 >> 1) of its 16
          uint8_t* d = dst + ((b * 2 + t) * NS + r) * 1024 + 16 * (32 * (q4 & 1) + 2 * n16) + 8 * (q4 >> 1);
          *reinterpret_cast<f16x4*>(d) = even[t];
          *reinterpret_cast<f16x4*>(d + 16) = odd[t];
        }
      } else {
        uint8_t* d = dst + (b * 2 * NS + 2 * r) * 1024 + 16 * ln;
        *reinterpret_cast<f16x8*>(d) = __builtin_shufflevector(even[0], even[1], 0, 1, 2, 3, 4, 5, 6, 7);
        *reinterpret_cast<f16x8*>(d + 1024) = __builtin_shufflevector(odd[0], odd[1], 0, 1, 2, 3, 4, 5, 6, 7);
      }
    }
  };

  // scores of a lane: RS = 32: position 32b + 8(i/4) + 4z + i%4 in sacc[b][0][i]; RS = 16: 32b + 16k + 4z + i in
  // sacc[b][k][i]
  constexpr int NK = kWide ? 1 : 2;
  Acc sacc[NU][NK];
  // raw scores of the step whose keys are in `src`
  auto scores = [&](const uint8_t* src, Acc (&x)[NU][NK]) __attribute__((always_inline)) {
    const uint8_t* kl = src + 16 * lane;
#pragma unroll
    for (int b = 0; b < NU; ++b)
#pragma unroll
      for (int k = 0; k < NK; ++k)
#pragma unroll
        for (int i = 0; i < NA; ++i) x[b][k][i] = 0.f;
#pragma unroll
    for (int t = 0; t < NQ; ++t)
#pragma unroll
      for (int b = 0; b < NU; ++b)
#pragma unroll
        for (int k = 0; k < NK; ++k) {
          const f16x8 kf = *reinterpret_cast<const f16x8*>(kl + (b * NT + k * NS + t) * 1024);
          if constexpr (kWide) x[b][k] = __builtin_amdgcn_mfma_f32_32x32x16_f16(kf, qf[t], x[b][k], 0, 0, 0);
          else x[b][k] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, qf[t], x[b][k], 0, 0, 0);
        }
  };
  // masks of the step at u
  auto mask = [&](int u, uint32_t none) __attribute__((always_inline)) {
    const int key0 = kKvUnit * u;
    if (key0 + NU * kKvUnit - 1 > pos_min || key0 < see_all || none) {
#pragma unroll
      for (int b = 0; b < NU; ++b)
#pragma unroll
        for (int k = 0; k < NK; ++k)
#pragma unroll
          for (int i = 0; i < NA; ++i) {
            const int key = key0 + 32 * b + (kWide ? 8 * (i >> 2) + 4 * z + (i & 3) : 16 * k + 4 * z + i);
            const bool seen = key <= pos && key >= low;
            sacc[b][k][i] = !seen ? -INFINITY : (none >> b) & 1u ? NAN : sacc[b][k][i];
          }
    }
  };
  // raw scores to exponents of p (base 2) under the current reference maximum; their largest
  auto exponents = [&]() __attribute__((always_inline)) {
    const float ref = m - kPExp;
    float mx = -INFINITY;
    if (__builtin_expect(any_far, 0)) {
#pragma unroll
      for (int b = 0; b < NU; ++b)
#pragma unroll
        for (int k = 0; k < NK; ++k)
#pragma unroll
          for (int i = 0; i < NA; ++i) {
            const float x = sacc[b][k][i];
            sacc[b][k][i] = far ? __fmaf_rn(x - m, c, kPExp) : __fmaf_rn(x, c, -ref);
            mx = fmaxf(mx, sacc[b][k][i]);
          }
      return mx;
    }
#pragma unroll
    for (int b = 0; b < NU; ++b)
#pragma unroll
      for (int k = 0; k < NK; ++k)
#pragma unroll
        for (int i = 0; i < NA; i += 2) {
          sacc[b][k][i] = __fmaf_rn(sacc[b][k][i], c, -ref);
          sacc[b][k][i + 1] = __fmaf_rn(sacc[b][k][i + 1], c, -ref);
          mx = fmaxf(mx, fmaxf(sacc[b][k][i], sacc[b][k][i + 1]));
        }
    return mx;
  };
  auto row_max = [](float v) { return kWide ? half_max(v) : quarter_max(v); };
  // the reference maximum moved to the largest of the raw scores, sums and outputs rescaled
  auto move_reference = [&]() __attribute__((always_inline)) {
    float mx = -INFINITY;
#pragma unroll
    for (int b = 0; b < NU; ++b)
#pragma unroll
      for (int k = 0; k < NK; ++k)
#pragma unroll
        for (int i = 0; i < NA; ++i) mx = fmaxf(mx, sacc[b][k][i]);
    const float f = kv_move(row_max(mx), c, m, far);
    any_far |= __any(far);
    l *= f;
#pragma unroll
    for (int r = 0; r < NO; ++r)
#pragma unroll
      for (int i = 0; i < NA; ++i) o[r][i] *= f;
  };
  f16x8 pf[NU][NSC / 8];      // RS = 32: 16 positions each; RS = 16: 32
  auto probabilities = [&]() __attribute__((always_inline)) {
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int b = 0; b < NU; ++b)
#pragma unroll
      for (int i = 0; i < NSC; i += 2) {
        const float p0 = exp2_hw(sacc[b][i / NA][i % NA]), p1 = exp2_hw(sacc[b][i / NA][i % NA + 1]);
        sum[(i >> 1) & 3] += p0 + p1;
        const f16x2 pr = __builtin_convertvector((f32x2){p0, p1}, f16x2);
        pf[b][i >> 3][i & 7] = pr[0];
        pf[b][i >> 3][(i & 7) + 1] = pr[1];
      }
    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
  };
  auto products = [&](const uint8_t* src) __attribute__((always_inline)) {
    const uint8_t* vl = src + 16 * lane;
#pragma unroll
    for (int b = 0; b < NU; ++b)
#pragma unroll
      for (int t = 0; t < NSC / 8; ++t)
#pragma unroll
        for (int r = 0; r < NO; ++r) {
          if (!kWide && r % 8 == 0) __builtin_amdgcn_sched_barrier(0);
          const f16x8 vf = *reinterpret_cast<const f16x8*>(vl + (b * 2 * NS + t * NO + r) * 1024);
          if constexpr (kWide) o[r] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf, pf[b][t], o[r], 0, 0, 0);
          else o[r] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, pf[b][t], o[r], 0, 0, 0);
        }
  };

  // Keys run one step ahead of values: while a step's probabilities are formed the next step's scores are
  // multiplied, and while its products run the operands of the keys two steps ahead and of the next
  // values are written.  Step i uses key buffer i & 1 and value buffer i & 1; one barrier per step.
  if (u0 < u1) {
    Step s1, s2, s3;      // the next step, the one after, the third
    {
      const Step s0 = locate(u0);
      load_keys(s0);
      load_values(s0);
      s1 = locate(u0 + NU);
      store_keys(key_lds0);
      store_values(u0, s0, value_lds0);
      load_keys(s1);
      store_keys(key_lds1);
      load_values(s1);
      s2 = locate(u0 + 2 * NU);
      load_keys(s2);
      __syncthreads();
      scores(key_lds0, sacc);
      mask(u0, s0.none);
      move_reference();
      exponents();
      __syncthreads();
    }
    // step u in buffers (kc, vc), the next step's in (kn, vn)
    auto step = [&](int u, uint8_t* kc, const uint8_t* kn, const uint8_t* vc, uint8_t* vn) __attribute__((always_inline)) {
      s3 = locate(u + 3 * NU);
      Acc next[NU][NK];
      probabilities();
      scores(kn, next);
      if (!kWide) __builtin_amdgcn_sched_barrier(0);
      store_keys(kc);                     // keys of u + 2*NU
      store_values(u + NU, s1, vn);
      load_keys(s3);
      load_values(s2);
      if (!kWide) __builtin_amdgcn_sched_barrier(0);
      products(vc);
      if (!kWide) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int b = 0; b < NU; ++b)
#pragma unroll
        for (int k = 0; k < NK; ++k) sacc[b][k] = next[b][k];
      mask(u + NU, s1.none);
      if (__builtin_expect(__any(exponents() > kSlack + kPExp), 0)) {
        scores(kn, sacc);      // the raw scores are gone
        mask(u + NU, s1.none);
        move_reference();
        exponents();
      }
      s1 = s2;
      s2 = s3;
      __syncthreads();
    };
    int u = u0;
    for (; u + 2 * NU < u1; u += 2 * NU) {
      step(u, key_lds0, key_lds1, value_lds0, value_lds1);
      step(u + NU, key_lds1, key_lds0, value_lds1, value_lds0);
    }
    if (u + NU < u1) {
      step(u, key_lds0, key_lds1, value_lds0, value_lds1);
      probabilities();
      products(value_lds1);
    } else {
      probabilities();
      products(value_lds0);
    }
  }

  l = kWide ? half_sum(l) : quarter_sum(l);
  m = kv_reference(m, c, far);
  if (!valid) return;
  const size_t at = (size_t)(it.q.row0 + tok) * a.Hq + h * a.G + g;
  // groups of four elements of the lane's row, and where they begin
  constexpr int NG = kWide ? 4 * NS : 2 * NS;
  auto group = [&](int k) __attribute__((always_inline)) {
    if constexpr (kWide) return float4{o[k / 4][4 * (k % 4)], o[k / 4][4 * (k % 4) + 1], o[k / 4][4 * (k % 4) + 2], o[k / 4][4 * (k % 4) + 3]};
    else return float4{o[k & ~1][2 * (k & 1)], o[k | 1][2 * (k & 1)], o[k & ~1][2 * (k & 1) + 1], o[k | 1][2 * (k & 1) + 1]};
  };
  auto place = [&](int k) { return kWide ? 8 * k + 4 * z : 32 * (k >> 1) + 8 * z + 4 * (k & 1); };
  if (it.splits == 1) {
    const bool any = l > 0.f || l != l;
    const float norm = any ? a.cache.v_gscale / l : 0.f;
    if (a.lse && z == 0) a.lse[at] = any ? kLn2 * (m + (__builtin_amdgcn_logf(l) - kPExp)) : -INFINITY;
#pragma unroll
    for (int k = 0; k < NG; ++k) {
      const float4 v = group(k);
      *reinterpret_cast<u32x2*>(a.out + at * D + place(k)) =
          u32x2{f32x2_to_bf16x2(v.x * norm, v.y * norm), f32x2_to_bf16x2(v.z * norm, v.w * norm)};
    }
  } else {
    const size_t slot = (size_t)(it.slot + it.split) * hkv + h;
    const int lrow = RS * wave + nrow;
    if (z == 0) {
      part.ml[slot * 2 * BM + lrow] = m;
      part.ml[slot * 2 * BM + BM + lrow] = l;
    }
#pragma unroll
    for (int k = 0; k < NG; ++k) *reinterpret_cast<float4*>(part.o + (slot * BM + lrow) * D + place(k)) = group(k);
  }
}

// ------------------------------------------------------------------------- combine
// Workgroup x joins, of shares, the tile x or the tile that share x leaves cut (one at most; it is another share's if it
// began before x), whichever are fewer, of items the x-th cut tile of its head: the launch is of the size of what can be
// cut, not of the step.  4096 requests of 40 positions, 32/8 heads, dimension 128: 443 us with the attention; a
// workgroup for each of their tiles, to find nearly all whole after a search of all lengths, 4140 us.  (64 of 40
// positions: 13.2 us by tiles, 14.6 us by shares.)
// One wave per row of a cut tile: lane i reads the maximum and sum of partial i, then D / 4 lanes take four
// elements each, 256 / D partials at a time, added in a fixed order.  Offsets into the partials fit 32 bits:
// there are at most 2 * 1024 of 16 rows or 2 * 1024 of 256.  Bound by latency (the schedule, the weights, the
// rows, one after the other): 7 us for 512 tiles of 8 rows with up to 9 partials each.
enum KvJoin { kItems, kTiles, kShares };
template <int D, KvJoin BY>
__global__ __launch_bounds__(256, 5) void kv_combine_kernel(KvAttentionProblem a, KvSchedule s, KvPartials part) {
  const int hkv = a.cache.kv_heads, lane = threadIdx.x & 63;
  KvRequest q;
  int h, tile, count;
  uint32_t first, step, odd;      // slots: first, then first + step*i - odd
  if (BY != kItems) {
    KvShare sh;
    KvWhere at;
    long long within;
    if (!kv_locate<BY == kTiles>(a, s, blockIdx.x + (BY == kShares ? 1 : 0), &sh, &at, &within)) return;
    q = at.q;
    // shares: the tile that holds the next share's first place.  Places of its first unit and its last.
    const long long step_length = kv_step(q, sh), nth = BY == kTiles ? within : div_i64(within, step_length);
    const long long start = BY == kTiles ? at.base + nth * step_length
                                         : (blockIdx.x + 1ll) * sh.chunk - (within - nth * step_length);
    const long long begin = start + (sh.aligned ? 0 : kSwitch);
    const long long i0 = div_i64(begin, sh.chunk), i1 = div_i64(begin + max(1, q.units) - 1, sh.chunk);
    if (i0 == i1 || (BY == kShares && i0 != blockIdx.x)) return;
    h = (int)div_i64(nth, q.tiles);
    tile = (int)(nth - (long long)h * q.tiles);
    count = (int)(i1 - i0) + 1;
    first = 2 * (uint32_t)i0 + 1;     // the share it begins in ends with it; the later ones begin with it
    step = 2;
    odd = 1;
  } else {
    KvItem it;
    if (!kv_find<true>(a, s, blockIdx.x / hkv, &it)) return;
    q = it.q;
    h = blockIdx.x % hkv;
    tile = it.tile;
    count = it.splits;
    first = (uint32_t)it.slot * hkv + h;
    step = hkv;
    odd = 0;
  }
  auto slot = [&](int i) { return first + step * (uint32_t)i - (i > 0 ? odd : 0u); };
  const int rows = min(s.bm, q.n * a.G - tile * s.bm);
  for (int row = 4 * blockIdx.y + (threadIdx.x >> 6); row < rows; row += 4 * gridDim.y) {
    const int grow = tile * s.bm + row;
    constexpr int LPR = D / 4, PER = 64 / LPR;      // lanes per partial row, partials per load
    constexpr int kLoads = D == 64 ? 4 : 8;         // loads in flight: 16, 16 or 8 partials
    const int sub = lane / LPR, d0 = 4 * (lane % LPR);
    float top = kNone, sum = 0.f;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    for (int i0 = 0; i0 < count; i0 += 64) {
      const int n = min(64, count - i0);
      f32x4 x[kLoads];
      auto load = [&](int j) {
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {
          const int i = j + k * PER + sub;
          x[k] = f32x4{0.f, 0.f, 0.f, 0.f};
          if (i < n) x[k] = *reinterpret_cast<const f32x4*>(part.o + ((slot(i0 + i) * s.bm + row) * D + d0));
        }
      };
      float mi = kNone, li = 0.f;
      if (lane < n) {
        const float* ml = part.ml + (slot(i0 + lane) * 2u * s.bm + row);
        mi = ml[0];
        li = ml[s.bm];
      }
      load(0);      // in flight while the weights are formed
      float most = fmaxf(mi, top);
#pragma unroll
      for (int off = 32; off >= 1; off >>= 1) most = fmaxf(most, __shfl_xor(most, off));
      const float f = exp2_hw(top - most), w = li != 0.f ? exp2_hw(mi - most) : 0.f;
      top = most;
      sum = sum * f + w * li;
      v *= f;
      for (int j = 0; j < n; j += kLoads * PER) {
        if (j > 0) load(j);
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {
          const float wk = __shfl(w, min(j + k * PER + sub, 63));
          v += wk * (wk != 0.f ? x[k] : f32x4{0.f, 0.f, 0.f, 0.f});      // an empty partial's outputs were not written
        }
      }
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) sum += __shfl_xor(sum, off);
#pragma unroll
    for (int off = LPR; off < 64; off <<= 1)
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += __shfl_xor(v[e], off);
    const bool any = sum > 0.f || sum != sum;
    const float norm = any ? a.cache.v_gscale / sum : 0.f;
    const int tok = grow / a.G, g = grow - tok * a.G;
    const size_t dst = (size_t)(q.row0 + tok) * a.Hq + h * a.G + g;
    if (sub == 0)
      *reinterpret_cast<u32x2*>(a.out + dst * D + d0) =
          u32x2{f32x2_to_bf16x2(v[0] * norm, v[1] * norm), f32x2_to_bf16x2(v[2] * norm, v[3] * norm)};
    if (a.lse && lane == 0) a.lse[dst] = any ? kLn2 * (top + (__builtin_amdgcn_logf(sum) - kPExp)) : -INFINITY;
  }
}

}  // namespace

size_t kv_attention_workspace(int32_t T, int32_t R, int32_t Hq, int32_t hkv, int32_t D, int64_t table_units) {
  if (T == 0 || R == 0) return 0;
  const Launches x = plan_launches(T, R, Hq / hkv, hkv, D, table_units);
  size_t bytes = 0;
  for (int i = 0; i < x.n; ++i) bytes = std::max(bytes, x.l[i].bytes);
  return bytes;
}

bool kv_attention_launchable(int32_t T, int32_t R, int32_t Hq, int32_t hkv, int32_t D, int64_t table_units) {
  return T == 0 || R == 0 || launchable(plan_launches(T, R, Hq / hkv, hkv, D, table_units));
}

moe_status_t launch_kv_attention(const KvAttentionProblem& problem, void* workspace, hipStream_t stream) {
  KvAttentionProblem a = problem;
  const int hkv = a.cache.kv_heads, D = a.cache.head_dim;
  const int64_t fill = a.fill ? std::min(((int64_t)a.T + 3) / 4, (int64_t)kCus) : 0;
  if (a.T == 0 || (a.R == 0 && !a.fill)) return MOE_OK;
  if (a.R == 0) {
    with_head_dim(D, [&](auto tag) {
      hipLaunchKernelGGL(kv_fill_kernel<decltype(tag)::value>, dim3((unsigned)fill), dim3(256), 0, stream, a);
    });
    return launch_status();
  }
  const Launches x = plan_launches(a.T, a.R, a.G, hkv, D, (int64_t)a.width * (a.cache.page_size / kKvUnit));
  for (int i = 0; i < x.n; ++i) {
    const Launch& p = x.l[i];
    KvPartials part{static_cast<float*>(workspace), nullptr};
    part.ml = reinterpret_cast<float*>(static_cast<char*>(workspace) + p.o_bytes);
    with_head_dim(D, [&](auto tag) {
      constexpr int DD = decltype(tag)::value;
      // few tiles: a wave per two rows, many: per eight, as most are found whole (5 prompts of 527 to 763
      // tokens, 2 heads: 28.8 against 35.8 us; a prompt of 2000, 32 heads: 73 against 70 us with twice as many)
      const int64_t most = p.s.bm / 8, join = std::max(p.join, (int64_t)1);
      const int64_t per_tile = std::max(std::min(most, (int64_t)4), std::min(most, 2048 / join));
      a.work_groups = (uint32_t)p.grid;
      const dim3 grid((unsigned)(p.grid + (i == 0 ? fill : 0))), rows((unsigned)join, (unsigned)per_tile);
      if (!p.shares) {
        if (DD != 256 && p.rs == 32)
          hipLaunchKernelGGL((kv_attention_tiles_kernel<DD == 256 ? 128 : DD, 8, 2, 32>), grid, dim3(512), 0, stream, a,
                             p.s, part);
        else
          hipLaunchKernelGGL((kv_attention_tiles_kernel<DD, 8, DD == 256 ? 1 : 2, 16>), grid, dim3(512), 0, stream, a,
                             p.s, part);
        if (p.join > 0) hipLaunchKernelGGL((kv_combine_kernel<DD, kItems>), rows, dim3(256), 0, stream, a, p.s, part);
      } else {
        if (p.whole)
          hipLaunchKernelGGL((kv_attention_rows_kernel<DD, 1, 8>), grid, dim3(512), 0, stream, a, p.s, part);
        else if (p.s.bm == 16)
          hipLaunchKernelGGL((kv_attention_rows_kernel<DD, 1, 4>), grid, dim3(256), 0, stream, a, p.s, part);
        else
          hipLaunchKernelGGL((kv_attention_rows_kernel<DD, 2, 4>), grid, dim3(256), 0, stream, a, p.s, part);
        if (p.join > 0 && p.join == p.tiles)
          hipLaunchKernelGGL((kv_combine_kernel<DD, kTiles>), rows, dim3(256), 0, stream, a, p.s, part);
        else if (p.join > 0)
          hipLaunchKernelGGL((kv_combine_kernel<DD, kShares>), rows, dim3(256), 0, stream, a, p.s, part);
      }
    });
    if (moe_status_t st = launch_status()) return st;
  }
  return MOE_OK;
}

}  // namespace moe
