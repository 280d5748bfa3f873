// Host build of the few-token layer's rules (csrc/few_rules.hpp), for
// tests/test_few_slices.py and tests/test_few_ticket_words.py.
#include "few_rules.hpp"

extern "C" {

int few_slice_step(int waited, int D) { return moe::few::slice_step(waited != 0, D); }
int few_ticket_number(unsigned word) { return moe::few::ticket_number(word); }
int few_adds_up(unsigned before, int D) { return moe::few::adds_up(before, D); }

}  // extern "C"
