// The order and the rows of the packed attention's workgroups (gfx950 and host).
#pragma once

namespace fp8sm {

// Row r of a prompt is token r / G and head r % G of the G query heads that share key
// head hk.  A lane's row of the tile that starts at r0 < rows, whose query it reads:
// behind the prompt's last row (not `ok`: nothing is seen or written) the tile's first,
// since other rows belong to other workgroups, which write there when o is q.
struct PackedRow {
  bool ok;
  int tok, head;
};
__host__ __device__ inline PackedRow packed_row(int r0, int i, int rows, int hk, int G) {
  const bool ok = r0 + i < rows;
  const int r = ok ? r0 + i : r0, tok = r / G;
  return PackedRow{ok, tok, hk * G + r - tok * G};
}

// A head's row tiles come with the last one (most tokens to see) first.  The list has
// the heads side by side, which leaves the short tiles of all heads for its end; with a
// multiple of eight heads each XCD reads the keys of its own ones.  More than 64 heads
// whose keys and values of a prompt (of average length, the host knows no other) outgrow the
// last-level cache (256 MB) follow each other, each XCD taking a contiguous part.  Causal
// heads of 128, us side by side and behind each other: 8320 tokens x 14 heads 240 and 327, x
// 56 (239 MB) 899 and 939, x 72 (307 MB) 1165 and 1196, x 80 (341 MB) 1305 and 1304, x 112
// 1892 and 1827; 4160 x 224 1112 and 1025, two of them x 192 1888 and 1795; 1000 x 80 36 and
// 45; 27 prompts of 300 x 128 301 and 408, x 256 617 and 867; 4 of 2000 x 256 (262 MB) 1385 and 1337.
// Up to 64 heads: 16640 x 40 (341 MB) 2468 and 2484, x 56 3511 and 3486, 33280 x 20 5039 and 5406.
__host__ __device__ inline bool heads_side_by_side(long long T, int prompts, int heads, int D) {
  return heads <= 64 || T / prompts * heads * D * 4 <= 5ll << 26;
}

}  // namespace fp8sm
