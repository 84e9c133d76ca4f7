// lores_scan_inst.cu -- the state scan's kernels of one key width and number of input planes
// (LORES_DK, LORES_NP), compiled once per pair so that the build runs in parallel.
#include "lores_scan.cuh"

namespace lores {
namespace scan {

template <int DK, int NP, bool DELTA>
static void fill(ScanKernels &t) {
  constexpr int NH = state_warps(DK);
  t.prep[NP - 1][DELTA][0] = scan_prep_kernel<DK, NP, DELTA, false>;
  t.prep[NP - 1][DELTA][1] = scan_prep_kernel<DK, NP, DELTA, true>;
  t.walk[NP - 1][DELTA][kForward] = scan_walk_kernel<DK, NP, DELTA, kForward, NH>;
  t.walk[NP - 1][DELTA][kRecompute] = scan_walk_kernel<DK, NP, DELTA, kRecompute, NH>;
  t.walk[NP - 1][DELTA][kReverse] = scan_walk_kernel<DK, NP, DELTA, kReverse, NH>;
  t.grads[NP - 1][DELTA] = scan_grads_kernel<DK, NP, DELTA>;
}

#define LORES_CAT3(a, b, c) a##b##_##c
#define LORES_CAT(a, b, c) LORES_CAT3(a, b, c)
void LORES_CAT(scan_kernels_, LORES_DK, LORES_NP)(ScanKernels &t) {
  fill<LORES_DK, LORES_NP, false>(t);
  fill<LORES_DK, LORES_NP, true>(t);
}

}  // namespace scan
}  // namespace lores
