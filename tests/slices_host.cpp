// Host build of the few-token layer's rules for the K slices of out (csrc/few_slices.hpp),
// for tests/test_few_slices.py.
#include "few_slices.hpp"

extern "C" {

int few_slice_step(int waited, int D) { return moe::few::slice_step(waited != 0, D); }
int few_adds_up(unsigned before, int D) { return moe::few::adds_up(before, D); }

}  // extern "C"
