"""Tickets of moe_layer_few from any word of its workspace (host check, no GPU): a call on the
same workspace may have put its data where tickets are counted. The kernel turns the word
that it counts up into a task by the rule of csrc/few_rules.hpp, times up to 8 tasks a ticket:
that has to be the task of a real ticket, or one past the last, never a negative number
(an address in front of the weights)."""
import ctypes
import os
import random
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sparse_mixture_experts_05_amd", "csrc")
# 256 experts + 512 pairs / 16 + 64 tokens / 16 units, 2^20 gated columns, 8 of them a task
MOST_TASKS = (256 + 32 + 4) * (1 << 20) // 8


@pytest.fixture(scope="module")
def number(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("few") / "slices_host.so")
    r = subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", f"-I{CSRC}",
                        os.path.join(ROOT, "tests", "slices_host.cpp"), "-o", out],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    L = ctypes.CDLL(out)
    L.few_ticket_number.argtypes = [ctypes.c_uint]
    return L.few_ticket_number


def first_task(n, batch):
    return int(np.int64(n * batch).astype(np.int32))  # the kernel's int


def check(number):
    rng = random.Random(1)
    words = [0, 1, 255, MOST_TASKS - 1, MOST_TASKS, 2 ** 31 - 1, 2 ** 31, 2 ** 32 - 1, 0x3f800000, 0xbf800000,
             0x7fc00000, 0xffffffff // 8, 2 ** 29, 2 ** 29 + 1] + [rng.getrandbits(32) for _ in range(2000)]
    for word in words:
        for batch in (1, 2, 4, 8):
            task = first_task(number(word), batch)
            if word * batch < MOST_TASKS:
                assert task == word * batch
            else:
                assert MOST_TASKS <= task <= 2 ** 31 - 1 - 8, (word, batch, task)


def test_any_word_is_a_task_or_none(number):
    check(number)


def test_check_finds_words_taken_as_they_are(number):
    with pytest.raises(AssertionError):
        check(lambda word: int(np.uint32(word).astype(np.int32)))
