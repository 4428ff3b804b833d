// The rows of a workgroup of the packed attention (gfx950 and host).
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

}  // namespace fp8sm
