"""The status word of the cache operators between streams."""
from __future__ import annotations

import random
import threading
import time

import pytest
import torch

import cacheutil as U
import tensor_command_execution_gb300 as T

pytestmark = pytest.mark.gpu


def test_no_status_bit_is_lost_between_streams():
    """Bits that operators on one stream set while another stream's word is read and cleared are all reported."""
    c = U.Cache("f32", [8, 8], 1, 8, 4, columns=2)
    bad_pages = c.tables.clone()
    bad_pages[1, 1] = c.pages
    bad_lengths = torch.tensor([8, 9], dtype=torch.int32, device="cuda")
    q, word = torch.randn(2, 1, 8, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    here, there = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    rng = random.Random(0)
    seen, stop, wrong = [0], threading.Event(), []

    def reader():
        try:
            while not stop.is_set():
                T.attention_decode(q, c.k, c.v, bad_pages, c.lengths, status=word, stream=there)
                try:
                    T.cache_status(word, stream=there)
                except T.CmdError as e:
                    seen[0] += "length" in str(e)
        except Exception as e:  # noqa: BLE001  (shown by the test)
            wrong.append(e)

    thread = threading.Thread(target=reader)
    thread.start()
    try:
        for i in range(2000):
            before = seen[0]
            with torch.cuda.stream(here):
                torch.cuda._sleep(rng.randrange(200_000))  # (anywhere in the reader's round)
            T.attention_decode(q, c.k, c.v, c.tables, bad_lengths, status=word, stream=here)
            here.synchronize()
            end = time.time() + 2.0
            while seen[0] == before and not wrong and time.time() < end:
                time.sleep(1e-5)
            assert not wrong and seen[0] > before, f"the bit of call {i} was never reported {wrong}"
    finally:
        stop.set()
        thread.join()
