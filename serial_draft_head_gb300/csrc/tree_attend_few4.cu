// tree_attend_few4.cu -- tree_attend_few4.cuh for heads of up to 64 elements, and the choice among
// its forms.
#include "tree_attend_few4.cuh"

namespace dspark {
namespace tree {

cudaError_t few4_setup128();
cudaError_t few4_launch128(const AttendArgs& a, bool two, bool alone, bool runs, cudaStream_t stream);

namespace {

cudaError_t setup64() {
  cudaError_t e = setup<64, 1, 16, false, false>();
  if (e == cudaSuccess) e = setup<64, 1, 16, false, true>();
  if (e == cudaSuccess) e = setup<64, 1, 16, true, false>();
  if (e == cudaSuccess) e = setup<64, 1, 16, true, true>();
  if (e == cudaSuccess) e = setup<64, 1, 4, true, false>();
  if (e == cudaSuccess) e = setup<64, 2, 12, false, false>();
  if (e == cudaSuccess) e = setup<64, 2, 12, false, true>();
  if (e == cudaSuccess) e = setup<64, 2, 12, true, false>();
  if (e == cudaSuccess) e = setup<64, 2, 12, true, true>();
  if (e == cudaSuccess) e = setup<64, 2, 4, true, false>();
  return e;
}

cudaError_t launch64(const AttendArgs& a, bool two, bool alone, bool runs, cudaStream_t stream) {
  const bool cap = a.softcap > 0.f;
  if (!runs) {
    if (two) return cap ? launch<64, 2, 12, false, true>(a, stream) : launch<64, 2, 12, false, false>(a, stream);
    return cap ? launch<64, 1, 16, false, true>(a, stream) : launch<64, 1, 16, false, false>(a, stream);
  }
  if (two) {
    if (cap) return launch<64, 2, 12, true, true>(a, stream);
    return alone ? launch<64, 2, 12, true, false>(a, stream) : launch<64, 2, 4, true, false>(a, stream);
  }
  if (cap) return launch<64, 1, 16, true, true>(a, stream);
  return alone ? launch<64, 1, 16, true, false>(a, stream) : launch<64, 1, 4, true, false>(a, stream);
}

// Whether a page holds each head's slots, and their scales, next to each other, in pieces
// that 16-byte copies take.
bool in_runs(const AttendArgs& a) {
  if (a.c.page.d % 16 != 0 || a.D % 64 != 0) return false;
  for (int v = 0; v < 2; ++v) {
    const Rows &x = a.c.x[v], &s = a.c.scale[v];
    if (x.slot != (uint32_t)a.D / 2 || s.slot != (uint32_t)a.D / 16) return false;
    if ((reinterpret_cast<uintptr_t>(s.p) | (uint64_t)s.head | s.page) % 16 != 0) return false;
  }
  return true;
}

}  // namespace

cudaError_t few4_setup(int D) { return padded_dim(D) == 64 ? setup64() : few4_setup128(); }

cudaError_t few4_launch(const AttendArgs& a, cudaStream_t stream) {
  // one tile of eight rows an item where the requests have no more on average
  const bool two = (int64_t)a.b.N * a.G > (int64_t)8 * a.b.B;
  // workers of four warps where there are two items a SM (64 heads on 8, 500 to 9,000
  // tokens, us with four / with a CTA's: 48 requests 76 / 93, 128 167 / 207; 16 requests 38 /
  // 39, 1 of 5,000 27 / 16, 19 of 32,767 156 / 144)
  const int64_t items = ((int64_t)a.b.N * a.G + 7) / 8 * a.Hkv;
  const bool alone = items < (int64_t)2 * a.n_cta;
  const bool runs = in_runs(a);
  return padded_dim(a.D) == 64 ? launch64(a, two, alone, runs, stream)
                               : few4_launch128(a, two, alone, runs, stream);
}

}  // namespace tree
}  // namespace dspark
