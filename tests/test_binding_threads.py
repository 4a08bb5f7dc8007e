"""Other Python threads run while an operator allocates and launches: with
switching by time all but off, a thread gets its turn only where a call gives
the interpreter up.  Calls of no rows allocate their outputs on the CPU."""
import sys
import threading
import time

import pytest
import torch


@pytest.mark.parametrize("name", ["logprobs", "append", "decode", "prefill"])
def test_an_operator_gives_up_the_interpreter(name):
    import qwen3_dense_decoder_gb300 as q3
    q3.build()
    kv, tab = torch.zeros(4, 2, 8, 2560, dtype=torch.uint8), torch.zeros(1, 2, dtype=torch.int32)
    row, gain, rope = torch.zeros(0, dtype=torch.int32), torch.ones(128, dtype=torch.bfloat16), torch.zeros(64, 64, 2)
    x, q, one = torch.zeros(0, 48 * 128), torch.zeros(0, 32, 128, dtype=torch.float16), torch.zeros(1, dtype=torch.int32)
    call = {"logprobs": lambda: q3.op_token_logprobs(x, None, 4), "append": lambda: q3.op_kv4_append(x, gain, gain, rope, row, row, tab, kv, 32),
            "decode": lambda: q3.op_kv4_decode_attention(q, row, row, tab, kv),
            "prefill": lambda: q3.op_kv4_prefill_attention(q, one, row, tab, kv)}[name]
    call()
    turns, stop, ready = [0], [False], threading.Event()

    def other():
        while not stop[0]:
            turns[0] += 1
            ready.set()
            time.sleep(0)

    interval = sys.getswitchinterval()
    t = threading.Thread(target=other)
    t.start()
    ready.wait()
    sys.setswitchinterval(1000)
    try:
        time.sleep(0.05)                                   # the other thread's waits now last that long too
        first = seen = turns[0]
        held = []                                          # freeing a tensor gives the interpreter up as well
        for _ in range(50000):
            held.append(call())
            seen = turns[0]
            if seen != first:
                break
    finally:
        sys.setswitchinterval(interval)
        stop[0] = True
        t.join()
    assert seen > first


def test_a_callers_outputs_keep_their_count():
    """Outputs that the caller passes are handed back: the same tensors, with no reference lost or kept."""
    import qwen3_dense_decoder_gb300 as q3
    q3.build()
    kv, tab, row = torch.zeros(4, 2, 8, 2560, dtype=torch.uint8), torch.zeros(1, 2, dtype=torch.int32), torch.zeros(0, dtype=torch.int32)
    one, q = torch.zeros(1, dtype=torch.int32), torch.zeros(0, 32, 128, dtype=torch.float16)
    out = torch.zeros(0, 32, 128, dtype=torch.float16)
    before = sys.getrefcount(out)
    for _ in range(100):
        assert q3.op_kv4_decode_attention(q, row, row, tab, kv, out=out) is out
        assert q3.op_kv4_prefill_attention(q, one, row, tab, kv, out=out) is out
        for bad in (torch.zeros(1, 32, 128, dtype=torch.float16), out.double()):
            with pytest.raises(ValueError):
                q3.op_kv4_decode_attention(q, row, row, tab, kv, out=bad)
    assert sys.getrefcount(out) == before
