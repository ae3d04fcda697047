// decode_ops.h -- the streaming core of the decode calls (hq_gemv, hq_moe_decode): a wave multiplies a
// few activation rows by a list of weight units (16 channels x 128 k), for every weight format with
// bf16 activations that these calls take.
//
// The work is bound by reading the packed weights once, so the core is a register ring: D units ahead
// are always in flight, each as plain vector loads (codes, scales, zeros) into registers, and every
// step of the loop issues exactly the same instructions -- units past the end are loads whose offset
// lies outside the buffer resource, which touch no memory and return 0. With no branch around a load
// the compiler's own wait counts stay exact; around a conditional load it falls back to waiting for
// everything, which empties the ring once per turn. Each piece was worth about a third: 14336 x 4096, M = 1,
// groups of 64: 13.4 us with plain loads unit by unit, 9.0 on the ring, 7.5 with the last turn free of loads
// (dead loads cost issue slots) and a ring of two; a deeper ring is slower wherever a wave has few units.
//
// Rows. The MFMA's A operand has 16 rows, its result D row 4 g + i, channel n in element i of lane
// 16 g + n. A row block is one of
//   AM = 1   one row (repeated; lane group 0's element 0 counts)
//   AM = 2   one row as a high and a low bf16 (MFMA rows 0 and 1: elements 0 and 1, added)
//   AM = 4   four rows at MFMA rows 0, 4, 8, 12: row g is element 0 of lane group g
//   AM = 6   two rows, each high (row 4 g) and low (row 4 g + 1), g = 0, 1
//   AM = 8   four rows, likewise
//   AM = 16  sixteen rows, all four elements
// so that for few rows the per-group scaling on the vector ALU (with the dequantization the larger
// part of the arithmetic) touches one element instead of four. The other MFMA rows repeat live
// ones and are dropped: rows do not mix in a matrix product.
// An item's activation rows reach LDS by direct copies, asked for with its weights.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "device_ops.h"
#include "layout.h"

namespace hq {

// INT4 with a scale per 128, 64 or 32 k, symmetric or with zero-points; MXFP4; 8-bit per channel.
enum DecFmt { DF_G128 = 0, DF_G128Z, DF_G64, DF_G64Z, DF_G32, DF_G32Z, DF_MXFP4, DF_INT8, DF_FP8 };

template <int F>
struct DecTraits {
  static constexpr bool kInt4 = F <= DF_G32Z;
  static constexpr bool kW8 = F == DF_INT8 || F == DF_FP8;
  static constexpr bool kAsym = F == DF_G128Z || F == DF_G64Z || F == DF_G32Z;
  static constexpr bool kFine = kInt4 && F >= DF_G64;
  static constexpr int kGroups = F == DF_G32 || F == DF_G32Z ? 4 : F == DF_G64 || F == DF_G64Z ? 2 : 1;
  static constexpr int kG = 128 / kGroups;
  static constexpr int kWLoads = kW8 ? 2 : 1;          // 1 KiB of codes each
  static constexpr int kUnit = kUnitBytes * kWLoads;   // code bytes of 16 channels x 128 k
  // bytes from one unit's scales to the next's
  static constexpr int kScaleStep = F == DF_MXFP4 ? 64 : kFine ? fine_meta_bytes(kG, kAsym) : 32;
  // vector loads per unit and tile; with CHAN, 8-bit weights' channel scales are among them
  template <bool CHAN>
  static constexpr int kLoads = kWLoads + (kW8 && !CHAN ? 0 : 1) + (kAsym ? 1 : 0);
};

// A layer's packed weights (one expert's, at w + e * expert_stride).
struct DecW {
  const uint8_t* w;
  size_t scales_off, zeros_off, expert_stride;
  int units;   // 128-k units per channel tile
};

// Which 16-byte chunk (8 k) of a unit's 128 k stands at chunk position 4 g + d of an LDS row, i.e. is
// fed by lane group g to MFMA d: the k order of the format's prepacked codes (layout.h).
template <int F>
__device__ __forceinline__ constexpr int dec_k_chunk(int at) {
  return DecTraits<F>::kFine ? ((at & 3) << 2) | (at >> 2) : at;
}

// LDS rows of a unit.
template <int AM>
constexpr int dec_rows() { return AM == 6 ? 4 : AM; }

// Row r's chunk at position p stands in slot p ^ key: with 256-byte rows every row starts in the same
// LDS bank, and unrotated the lanes of one read would all meet there.
template <int AM>
__device__ __forceinline__ int dec_key(int r) {
  return AM == 16 ? (((r & 7) << 1) | ((r >> 3) & 1)) : AM == 8 ? (r >> 1) : r;
}

// The LDS row that lane l feeds to the MFMA (its row l & 15).
template <int AM>
__device__ __forceinline__ int dec_lds_row(int lane) {
  const int r = lane & 15;
  return AM == 1 ? 0 : AM == 2 ? (r & 1) : AM == 4 ? (r >> 2) : AM == 6 ? (((r >> 2) & 1) * 2 + (r & 1)) : AM == 8 ? ((r >> 2) * 2 + (r & 1)) : r;
}

typedef __amdgpu_buffer_rsrc_t rsrc_t;

// Buffer resource over `bytes` bytes at p (wave-uniform): loads past them return 0 and touch nothing.
__device__ __forceinline__ rsrc_t dec_rsrc(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, int(bytes), 0x00027000);
}
// 16 bytes a lane from a buffer to LDS (lane i's land at lds + 16 i; lds is wave-uniform). The buffer
// form, not the global one: the compiler takes a global copy to LDS for a flat access, and while one
// is open it turns every wait for a vector load into a wait for all of them.
__device__ __forceinline__ void dec_lds_copy(rsrc_t r, uint32_t at, uint8_t* lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16, int(at), 0, 0, 0);
}
constexpr uint32_t kDecOutside = 0x7FFFFFFFu;   // past every resource here (they stay below 2^31 bytes)
constexpr int kNT = 2;                          // cache hint: streamed once

// One tile's buffers: codes and scales (fine groups: scales and zeros), zeros. Neighbouring tiles of
// one expert may share them.
template <int F>
struct DecTile {
  rsrc_t codes, scales, zeros;
};

// Buffers over `tiles` tiles from tile nt on of the expert at w. CHAN: 8-bit weights' channel scales too.
template <int F, bool CHAN = false>
__device__ __forceinline__ DecTile<F> dec_tile(const DecW& W, const uint8_t* w, int nt, int tiles = 1) {
  using T = DecTraits<F>;
  DecTile<F> t;
  const size_t at = size_t(nt) * W.units;
  t.codes = dec_rsrc(w + at * T::kUnit, uint32_t(tiles) * W.units * T::kUnit);
  if constexpr (!T::kW8) t.scales = dec_rsrc(w + W.scales_off + at * T::kScaleStep, uint32_t(tiles) * W.units * T::kScaleStep);
  else if constexpr (CHAN) t.scales = dec_rsrc(w + W.scales_off + size_t(nt) * 64, uint32_t(tiles) * 64);
  if constexpr (F == DF_G128Z) t.zeros = dec_rsrc(w + W.zeros_off + at * 8, uint32_t(tiles) * W.units * 8);
  return t;
}

// A unit in flight: the lane's codes and its channel's scales and zeros, as loaded.
template <int F>
struct DecUnit {
  u32x4 q[DecTraits<F>::kWLoads];
  uint32_t s[DecTraits<F>::kGroups == 4 ? 2 : 1];
  uint32_t z;
};

// Load unit u of a tile, counted from its buffers' start (live false: nothing is read). CHAN: 8-bit
// weights' channel scales from the buffer's tile nt.
template <int F, bool CHAN>
__device__ __forceinline__ void dec_load(DecUnit<F>& v, const DecTile<F>& t, int u, int nt, bool live, int lane) {
  using T = DecTraits<F>;
  const uint32_t at = live ? uint32_t(u) * T::kUnit : kDecOutside - 16 * 64;
#pragma unroll
  for (int i = 0; i < T::kWLoads; ++i)
    v.q[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(t.codes, int(at + 1024 * i + 16 * lane), 0, kNT));
  if constexpr (!T::kW8) {
    const uint32_t ms = live ? uint32_t(u) * T::kScaleStep : kDecOutside - 4096;
    const int n = lane & 15;
    if constexpr (F == DF_MXFP4) v.s[0] = __builtin_amdgcn_raw_buffer_load_b8(t.scales, int(ms + lane), 0, 0);
    else if constexpr (T::kGroups == 1) v.s[0] = __builtin_amdgcn_raw_buffer_load_b16(t.scales, int(ms + 2 * n), 0, 0);
    else if constexpr (T::kGroups == 2) v.s[0] = __builtin_amdgcn_raw_buffer_load_b32(t.scales, int(ms + 4 * n), 0, 0);
    else {
      const auto s2 = __builtin_amdgcn_raw_buffer_load_b64(t.scales, int(ms + 8 * n), 0, 0);
      v.s[0] = s2[0];
      v.s[1] = s2[1];
    }
    if constexpr (F == DF_G128Z)
      v.z = __builtin_amdgcn_raw_buffer_load_b8(t.zeros, int((live ? uint32_t(u) * 8 : kDecOutside - 4096) + (n >> 1)), 0, 0);
    else if constexpr (F == DF_G64Z)
      v.z = __builtin_amdgcn_raw_buffer_load_b8(t.scales, int(ms + fine_scale_bytes(64) + n), 0, 0);
    else if constexpr (F == DF_G32Z)
      v.z = __builtin_amdgcn_raw_buffer_load_b16(t.scales, int(ms + fine_scale_bytes(32) + 2 * n), 0, 0);
  } else if constexpr (CHAN) {
    v.s[0] = __builtin_amdgcn_raw_buffer_load_b32(t.scales, int(live ? 64 * nt + 4 * (lane & 15) : kDecOutside - 4096), 0, 0);
  }
}

// Elements of the result that count, and how they come out of an MFMA tile.
template <int AM>
constexpr int dec_elems() { return AM == 16 ? 4 : 1; }
template <int AM>
__device__ __forceinline__ float dec_elem(const f32x4& d, int i) {
  return AM == 2 || AM == 6 || AM == 8 ? d[0] + d[1] : d[i];
}

// acc += the unit's product with the A operand af; rs: the row sums of its groups (INT4).
//
// INT4: sum_k x (q - z) of a group is formed as sum_k x (128 + q) -- 128 + q is one bit-select per pair of
// codes, exact in bf16 -- less (128 + z) sum_k x, the row sums coming from the MFMA against ones
// (shared by a wave's tiles). Scales multiply the fp32 partial sum of each group: folded into the
// bf16 operand they would be rounded once per weight (half a step, 2^-8 of each).
template <int F, int AM>
__device__ __forceinline__ void dec_mul(f32x4& acc, const u32x4 (&af)[4], const float (&rs)[DecTraits<F>::kGroups][dec_elems<AM>()],
                                        const DecUnit<F>& v, int lane) {
  using T = DecTraits<F>;
  if constexpr (T::kInt4) {
    constexpr int per = 4 / T::kGroups;   // MFMAs per group
#pragma unroll
    for (int g = 0; g < T::kGroups; ++g) {
      f32x4 part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int d = g * per; d < (g + 1) * per; ++d)
        part = mfma_bf16(__builtin_bit_cast(bf16x8, af[d]), dequant_int4x8_offset128(v.q[0][d]), part);
      const uint32_t sw = v.s[g >> 1];
      const float s = __uint_as_float((g & 1) ? (sw & 0xFFFF0000u) : (sw << 16));
      // 128 + z: 128.0's mantissa step at bit 16 is 1
      uint32_t z = 8;
      if constexpr (F == DF_G128Z) z = (v.z >> (4 * (lane & 1))) & 0xF;
      else if constexpr (T::kAsym) z = (v.z >> (4 * g)) & 0xF;
      const float zo = __uint_as_float(0x43000000u | (z << 16));
#pragma unroll
      for (int i = 0; i < dec_elems<AM>(); ++i) acc[i] = fmaf(s, fmaf(-zo, rs[g][i], dec_elem<AM>(part, i)), acc[i]);
    }
  } else {
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      bf16x8 b;
      if constexpr (F == DF_MXFP4) b = dequant_fp4x8_scaled(v.q[0][d], e8m0_to_f32(v.s[0]));
      else b = dequant_w8_step<F == DF_FP8>(v.q[0], v.q[1], d);
      acc = mfma_bf16(__builtin_bit_cast(bf16x8, af[d]), b, acc);
    }
  }
}

// The value of element i of an accumulator after the last unit (INT4 adds the halves per group).
template <int F, int AM>
__device__ __forceinline__ float dec_value(const f32x4& acc, int i) {
  if constexpr (DecTraits<F>::kInt4) return acc[i];
  else return dec_elem<AM>(acc, i);
}

template <int F, int AM>
__device__ __forceinline__ void dec_row_sums(const u32x4 (&af)[4], float (&rs)[DecTraits<F>::kGroups][dec_elems<AM>()]) {
  using T = DecTraits<F>;
  if constexpr (T::kInt4) {
    const bf16x8 ones = __builtin_bit_cast(bf16x8, u32x4{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u});
    constexpr int per = 4 / T::kGroups;
#pragma unroll
    for (int g = 0; g < T::kGroups; ++g) {
      f32x4 r = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int d = g * per; d < (g + 1) * per; ++d) r = mfma_bf16(__builtin_bit_cast(bf16x8, af[d]), ones, r);
#pragma unroll
      for (int i = 0; i < dec_elems<AM>(); ++i) rs[g][i] = dec_elem<AM>(r, i);
    }
  }
}

// Copies of an item's activation rows (four 256-byte rows each), and a wave's LDS: D items' rows.
template <int AM>
constexpr int dec_copies() { return (dec_rows<AM>() + 3) / 4; }
template <int AM, int D>
constexpr int dec_wave_lds() { return D * dec_copies<AM>() * 1024; }

// The wave's loop over n items. An item is a unit of the wave's NT tiles:
//   item(i)     called before item i is loaded
//   tile(t)     the DecTile of its tile t                      (wave-uniform)
//   unit(i, t)  its unit, counted from that tile's buffers' start (wave-uniform)
//   row(i, r)   byte offset in `rows` of LDS row r's first k of the item (any lane's r)
//   done(i, units)  called after item i's products were added, with its units as loaded
// Items past the last are asked for with i clamped to n - 1.
template <int F, int AM, int NT, int D, bool CHAN = false, class Item, class Tile, class Unit, class Row, class Done>
__device__ __forceinline__ void dec_stream(int n, rsrc_t rows, uint8_t* lds, int lane, f32x4 (&acc)[NT], Item&& item, Tile&& tile,
                                           Unit&& unit, Row&& row, Done&& done) {
  using T = DecTraits<F>;
  constexpr int ROWS = dec_rows<AM>();
  constexpr int NA = dec_copies<AM>();
  constexpr int PER = NT * T::template kLoads<CHAN>;   // vector loads per item
  static_assert(D * (PER + NA) < 64, "vmcnt range");
  if (n <= 0) return;

  // Ask for item i, into slot j: its rows, then its tiles' units.
  DecUnit<F> ring[D][NT];
  auto load = [&](int j, int i) __attribute__((always_inline)) {
    const int ic = min(i, n - 1);
    item(ic);
#pragma unroll
    for (int a = 0; a < NA; ++a) {
      const int r = (4 * a + (lane >> 4)) % ROWS;   // fewer than four rows: again
      const int c = dec_k_chunk<F>((lane & 15) ^ dec_key<AM>(r));
      dec_lds_copy(rows, uint32_t(row(ic, r)) + 16 * c, lds + (j * NA + a) * 1024);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) dec_load<F, CHAN>(ring[j][t], tile(t), unit(ic, t), t, i < n, lane);
    // Keep the issue order as written, before the loop as in it: the wait before a slot's first use has to
    // hold for both ways into the loop, and with another order before it that would be a wait for everything.
    asm volatile("" ::: "memory");
  };
#pragma unroll
  for (int j = 0; j < D; ++j) load(j, j);
  const int rr = dec_lds_row<AM>(lane);
  const int blocks = (n + D - 1) / D;
  // D items from b * D on; MORE: refill each slot as it is used up.
  auto turn = [&](int b, auto more) __attribute__((always_inline)) {
    constexpr bool MORE = decltype(more)::value;
#pragma unroll
    for (int j = 0; j < D; ++j) {
      const int i = b * D + j;
      // the item's rows have landed: only its own loads and the items asked for after it may be open
      const int after = MORE ? D - 1 : D - 1 - j;
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"(PER + after * (PER + NA)) : "memory");
      if (MORE || i < n) {   // every turn but the last is a whole one
        const uint8_t* base = lds + j * NA * 1024 + rr * 256;
        u32x4 af[4];
#pragma unroll
        for (int d = 0; d < 4; ++d)
          af[d] = *reinterpret_cast<const u32x4*>(base + 16 * ((4 * (lane >> 4) + d) ^ dec_key<AM>(rr)));
        float rs[T::kGroups][dec_elems<AM>()];
        dec_row_sums<F, AM>(af, rs);
#pragma unroll
        for (int t = 0; t < NT; ++t) dec_mul<F, AM>(acc[t], af, rs, ring[j][t], lane);
        done(i, ring[j]);
      }
      if constexpr (MORE) {
        // every read of the slot's rows has completed before its next contents are asked for
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        load(j, i + D);
      }
    }
  };
  for (int b = 0; b + 1 < blocks; ++b) turn(b, std::true_type{});
  turn(blocks - 1, std::false_type{});
  // nothing of this wave may still be on its way into LDS when the caller uses it for something else
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
}

}  // namespace hq
