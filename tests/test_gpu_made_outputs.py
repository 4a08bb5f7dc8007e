"""What the asynchronous operators make for a caller is made as torch makes it where
something other than the allocator has a part in that: new memory is filled where
deterministic algorithms ask for it, and dispatch modes and profilers see it made."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q3():
    import qwen3_dense_decoder_gb300 as q3
    q3.build()
    return q3


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def calls(q3):
    """Every operator once; each gives the tensors that it made."""
    x = torch.randn(5, 100, device="cuda")
    gain = torch.ones(100, device="cuda").bfloat16()
    codes, scales = q3.op_i8_quantize(x)
    kv = torch.zeros(4, 2, 2, q3.KV4_TILE, dtype=torch.uint8, device="cuda")
    qkv, tables, pos, slot = torch.randn(5, 8 * 128, device="cuda"), ints(0, 1, 2, 3).view(1, 4), ints(0, 1, 2, 3, 4), ints(0, 0, 0, 0, 0)
    ones = torch.ones(128, device="cuda").bfloat16()
    rope = q3.rope_table(128, 1e6)
    q = q3.op_kv4_append(qkv, ones, ones, rope, pos, slot, tables, kv, 4)
    return {
        "i8_quantize": lambda: q3.op_i8_quantize(x),
        "i8_norm": lambda: q3.op_i8_norm(x, gain, delta=x),
        "i8_swiglu": lambda: q3.op_i8_swiglu(x),
        "i8_matmul": lambda: (q3.op_i8_matmul(codes, scales, codes, scales),),
        "kv4_append": lambda: (q3.op_kv4_append(qkv, ones, ones, rope, pos, slot, tables, kv, 4),),
        "kv4_decode_attention": lambda: (q3.op_kv4_decode_attention(q, pos, slot, tables, kv),),
        # three of five rows belong to a sequence; the others are left as they were
        "kv4_prefill_attention": lambda: (q3.op_kv4_prefill_attention(q, ints(0, 3), ints(0), tables, kv),),
        "token_logprobs": lambda: q3.op_token_logprobs(x, ints(1, 2, 3, 4, 5), 3),
    }


NAMES = ("i8_quantize", "i8_norm", "i8_swiglu", "i8_matmul", "kv4_append", "kv4_decode_attention", "kv4_prefill_attention", "token_logprobs")
MADE = {"i8_quantize": 2, "i8_norm": 3, "i8_swiglu": 2, "i8_matmul": 1, "kv4_append": 1, "kv4_decode_attention": 1, "kv4_prefill_attention": 2,
        "token_logprobs": 4}                               # (the prefill attention's workspace too)


@pytest.fixture
def deterministic():
    torch.use_deterministic_algorithms(True)
    yield
    torch.use_deterministic_algorithms(False)


def test_new_memory_is_filled_where_that_is_asked_for(q3, deterministic):
    assert torch.utils.deterministic.fill_uninitialized_memory
    f = calls(q3)
    for _ in range(3):
        rows = f["kv4_prefill_attention"]()[0]
        assert not torch.isnan(rows[:3]).any() and torch.isnan(rows[3:]).all()


class Seen(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.made = 0

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        self.made += func in (torch.ops.aten.empty.memory_format, torch.ops.aten.empty_strided.default)
        return func(*args, **(kwargs or {}))


@pytest.mark.parametrize("name", NAMES)
def test_a_dispatch_mode_sees_what_is_made(q3, name):
    f = calls(q3)[name]
    want = f()
    extra = 2 if name == "kv4_prefill_attention" else 1 if name == "token_logprobs" else 0     # the call's own torch.tensor
    with Seen() as none:
        for _ in range(extra):
            ints(1)
    with Seen() as seen:
        got = f()
    assert seen.made - none.made == MADE[name]
    if name != "kv4_prefill_attention":
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    else:
        assert torch.equal(got[0][:3], want[0][:3])


def test_a_profiler_sees_what_is_made(q3):
    f = calls(q3)["i8_norm"]
    f()
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CPU]) as p:
        f()
    made = sum(e.count for e in p.key_averages() if e.key in ("aten::empty", "aten::empty_strided"))
    assert made >= 3


@pytest.mark.parametrize("name", NAMES)
def test_the_same_either_way(q3, name, deterministic):
    f = calls(q3)[name]
    filled = [t.clone() for t in f()]
    torch.use_deterministic_algorithms(False)
    plain = f()
    for a, b in zip(filled, plain):
        assert a.dtype == b.dtype and a.shape == b.shape and a.device == b.device and b.requires_grad == a.requires_grad
        a, b = (a[:3], b[:3]) if name == "kv4_prefill_attention" else (a, b)
        assert torch.equal(a, b)
