// lores_scan_inst.cu -- the state scan's kernels of one key width and number of input planes
// (LORES_DK, LORES_NP), compiled once per pair so that the build runs in parallel.
#include "lores_scan.cuh"

namespace lores {
namespace scan {

template <int DK, int NP>
static void fill(ScanKernels &t) {
  constexpr int TWO = DK >= 32 ? 2 : 1;          // half a 16-column state has no whole k-step
  t.prep[NP - 1][0][0] = scan_prep_kernel<DK, NP, false, false>;
  t.prep[NP - 1][0][1] = scan_prep_kernel<DK, NP, false, true>;
  t.prep[NP - 1][1][0] = scan_prep_kernel<DK, NP, true, false>;
  t.prep[NP - 1][1][1] = scan_prep_kernel<DK, NP, true, true>;
  t.chain[NP - 1][0][0][0] = scan_chain_kernel<DK, NP, false, false, 1>;
  t.chain[NP - 1][0][0][1] = scan_chain_kernel<DK, NP, false, false, TWO>;
  t.chain[NP - 1][0][1][0] = scan_chain_kernel<DK, NP, false, true, 1>;
  t.chain[NP - 1][0][1][1] = scan_chain_kernel<DK, NP, false, true, TWO>;
  t.chain[NP - 1][1][0][0] = scan_chain_kernel<DK, NP, true, false, 1>;
  t.chain[NP - 1][1][0][1] = scan_chain_kernel<DK, NP, true, false, TWO>;
  t.chain[NP - 1][1][1][0] = scan_chain_kernel<DK, NP, true, true, 1>;
  t.chain[NP - 1][1][1][1] = scan_chain_kernel<DK, NP, true, true, TWO>;
  t.reverse[NP - 1][0][0] = scan_reverse_kernel<DK, NP, false, 1>;
  t.reverse[NP - 1][0][1] = scan_reverse_kernel<DK, NP, false, TWO>;
  t.reverse[NP - 1][1][0] = scan_reverse_kernel<DK, NP, true, 1>;
  t.reverse[NP - 1][1][1] = scan_reverse_kernel<DK, NP, true, TWO>;
  t.grads[NP - 1][0] = scan_grads_kernel<DK, NP, false>;
  t.grads[NP - 1][1] = scan_grads_kernel<DK, NP, true>;
}

#define LORES_CAT3(a, b, c) a##b##_##c
#define LORES_CAT(a, b, c) LORES_CAT3(a, b, c)
void LORES_CAT(scan_kernels_, LORES_DK, LORES_NP)(ScanKernels &t) { fill<LORES_DK, LORES_NP>(t); }

}  // namespace scan
}  // namespace lores
