"""What the calls through the extension module do when the library's call fails, and that
other threads run beside it (needs a B200)."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import reciprocal_nearest_neighbour_b200 as rnn
from test_gpu_q8 import filled, gen_of, ints, normal

pytestmark = pytest.mark.gpu

HF = torch.float16
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NAMES = ("rnn_kv_read_q8", "rnn_attn_decode_q8", "rnn_attn_decode_q8_workspace_size",
         "rnn_attn_decode_shared", "rnn_attn_decode_shared_workspace_size", "rnn_kv_append_q8")


def address(f):
    return ctypes.cast(f, ctypes.c_void_p).value


@pytest.fixture
def entry():
    """Puts a function in the place of the library's calls, until the test's end."""
    lib, fast = rnn._lib.load(), rnn._lib.load_fast()

    def put(f):
        fast.bind(*(address(getattr(lib, n) if f is None or n.endswith("_size") else f)
                    for n in NAMES))

    yield put
    put(None)


def calls():
    """The four calls, on small inputs, and the tensors that they write."""
    g = gen_of(3)
    kc, vc, scales, _, _ = filled(g, "int8", 3, 16, 2, 64)
    k16, v16 = (normal(g, (3, 16, 2, 64), HF) for _ in range(2))
    q, k, v = (normal(g, (5, h, 64), HF) for h in (4, 2, 2))
    one = normal(g, (1, 4, 64), HF)
    inv = torch.ones(32, dtype=torch.float64, device="cuda")
    tab = ints([[0, 1]])
    outs = [torch.full((1, 4, 64), 7.0, dtype=HF, device="cuda") for _ in range(2)]
    read = [torch.full((5, 2, 64), 7.0, dtype=HF, device="cuda") for _ in range(2)]
    todo = {
        "kv_append_q8": lambda m, n: m(k, v, kc, vc, scales, tab, ints([0]), ints([0, 5]),
                                       **n(q=q, inv_freq=inv, positions=None, paired=False,
                                           with_k=False, q_out=q, k_out=k)),
        "kv_read_q8": lambda m, n: m(kc, vc, scales, tab, ints([0, 5]), 5, n.dtype,
                                     **n(start=None, k_out=read[0], v_out=read[1])),
        "attn_decode_q8": lambda m, n: m(one, kc, vc, scales, tab, ints([20]),
                                         **n(scale=0.25, with_lse=False, out=outs[0], workspace=None)),
        "attn_decode_shared": lambda m, n: m(one, k16, v16, ints([2]), ints([9]), tab, ints([20]),
                                             **n(scale=0.25, with_lse=False, out=outs[1],
                                                 workspace=None)),
    }
    return todo, [q, k, kc, vc, scales, *outs, *read]


class Named:
    """Keyword arguments of the package's function."""
    dtype = HF

    def __call__(self, **kw):
        return kw


@pytest.mark.parametrize("name", ["kv_append_q8", "kv_read_q8", "attn_decode_q8", "attn_decode_shared"])
@pytest.mark.parametrize("code", [4, 6])
def test_a_failed_call_is_not_made_again(entry, name, code):
    """A status of the library reaches the caller; nothing runs a second time (rows rotated
    in place would be turned twice)."""
    todo, written = calls()
    before = [t.clone() for t in written]
    made = []

    @ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p)
    def fails(args, stream):
        made.append(args)
        return code

    entry(fails)
    with pytest.raises(rnn.RNNError) as e:
        todo[name](getattr(rnn, name), Named())
    assert e.value.name == rnn._lib.STATUS[code] and len(made) == 1
    torch.cuda.synchronize()
    for t, was in zip(written, before):
        assert torch.equal(t.view(torch.uint8), was.view(torch.uint8))
    entry(None)
    assert todo[name](getattr(rnn, name), Named()) is not None


@pytest.mark.parametrize("name", ["kv_append_q8", "kv_read_q8", "attn_decode_q8", "attn_decode_shared"])
def test_the_interpreter_is_free_during_the_call(entry, name):
    """In the library's place a function that says whether its thread holds the lock."""
    todo, _ = calls()
    fast = rnn._lib.load_fast()
    entry(ctypes.pythonapi.PyGILState_Check)
    seen = []

    def positional(*args, **kw):
        order = {"kv_append_q8": ("q", "inv_freq", "positions", "paired", "with_k", "q_out", "k_out"),
                 "kv_read_q8": ("start", "k_out", "v_out")}.get(
                     name, ("scale", "with_lse", "out", "workspace"))
        args = list(args)
        if name == "kv_read_q8":
            args[-1] = False                 # bf16 or not
        seen.append(getattr(fast, name)(*args, *(kw[x] for x in order)))

    todo[name](positional, Named())
    # 0, and so the call's result; 1 is a status
    assert seen[0] is not None and not isinstance(seen[0], int)


LEFT_BEHIND = """
import torch, reciprocal_nearest_neighbour_b200 as rnn
x = torch.ones(4, 2, 64, device="cuda").half()
cache = torch.zeros(2, 16, 2, 64, device="cuda").half()
i = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")
args = (x, x, cache, cache.clone(), i(0, 1)[None], i(0), i(0, 4))
rnn.kv_append(*args)
ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
torch.cuda.synchronize()
s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
failed = False
try:
    with torch.cuda.stream(s):
        g.capture_begin(capture_error_mode="thread_local")
        try:
            rnn.workspace_status(ws)         # waits for its stream, which a capture cannot
        except rnn.RNNError as e:
            failed = e.name == "RNN_ECUDA"
        finally:
            g.capture_end()
except RuntimeError:
    pass                                     # the capture is lost
assert failed
rnn.kv_append(*args)
torch.cuda.synchronize()
print("the next call is fine")
"""


def test_a_failed_call_leaves_nothing_for_the_next():
    """An error of the runtime that one call reported is not reported again by another."""
    r = subprocess.run([sys.executable, "-c", LEFT_BEHIND], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "the next call is fine" in r.stdout, r.stdout + r.stderr


def good_calls():
    """Arguments by position, of calls that are served."""
    g = gen_of(3)
    kc, vc, scales, _, _ = filled(g, "int8", 3, 16, 2, 64)
    k16, v16 = (normal(g, (3, 16, 2, 64), HF) for _ in range(2))
    q, k, v = (normal(g, (5, h, 64), HF) for h in (4, 2, 2))
    inv = torch.ones(16, dtype=torch.float64, device="cuda")
    at = ints([[1, 2]] * 5)
    tab, cu, two, one = ints([[0, 1], [2, 2]]), ints([0, 2, 5]), ints([3, 4]), ints([9])
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    return {
        "kv_append_q8": [k, v, kc, vc, scales, tab, two, cu, q, inv, at, False, True,
                         torch.empty_like(q), torch.empty_like(k)],
        "kv_read_q8": [kc, vc, scales, tab, cu, 5, False, two, torch.empty_like(k),
                       torch.empty_like(k)],
        "attn_decode_q8": [q[:2], kc, vc, scales, tab, two, 0.25, True, torch.empty_like(q[:2]), ws],
        "attn_decode_shared": [q[:2], k16, v16, one, one, tab, two, 0.25, True,
                               torch.empty_like(q[:2]), ws],
    }


def worse(x):
    """Forms of an argument that its call cannot take as it is."""
    if isinstance(x, bool):
        return {"an int": 1, "none": None}
    if isinstance(x, float):
        return {"negative": -1.0, "nan": float("nan"), "too large": 1e39, "zero": 0.0, "text": "1"}
    if isinstance(x, int):
        return {"negative": -1, "a float": 5.0, "more": 6, "beyond 64 bits": 1 << 70}
    bad = {"no tensor": 3, "a list": [1], "on the host": x.cpu(), "of another type": x.to(torch.complex64),
           "a dimension more": x[None], "a dimension less": x[0], "nothing": x[:0]}
    if x.dim() > 1 or x.dtype != torch.uint8:
        bad["one less"] = x[:-1]
        if x.numel() > 1:
            bad["not contiguous"] = torch.stack([x, x], -1)[..., 0]
    if x.dim() >= 2:
        bad["one wider"] = torch.cat([x, x[..., :1]], -1)
        bad["a row less"] = x[:, :-1]
    if x.dim() >= 3 and x.dtype != torch.float32:
        room = torch.zeros(x.numel() + 64, dtype=x.dtype, device="cuda")
        bad["off its boundary"] = room[1:1 + x.numel()].view(x.shape)
        bad["strides of 4"] = torch.zeros(*x.shape[:-1], x.shape[-1] + 4, dtype=x.dtype,
                                          device="cuda")[..., :x.shape[-1]]
    return bad


# What a call takes after all: longer or shorter rows of the page table, fewer pairs to rotate,
# one column of positions; a workspace whose size the library refuses itself.
ALLOWED = {
    "kv_append_q8": {(5, "one wider"), (5, "a row less"), (9, "one less"), (10, "a row less")},
    "kv_read_q8": {(3, "one wider"), (3, "a row less")},
    "attn_decode_q8": {(4, "one wider"), (4, "a row less"), (9, "nothing")},
    "attn_decode_shared": {(5, "one wider"), (5, "a row less"), (10, "nothing")},
}


@pytest.mark.parametrize("name", ["kv_append_q8", "kv_read_q8", "attn_decode_q8", "attn_decode_shared"])
def test_unusual_arguments_do_not_reach_the_library(entry, name):
    """Each argument in turn in a form that does not fit the others.  In the library's place a
    function that launches nothing."""
    fast, good = rnn._lib.load_fast(), good_calls()[name]
    made = []

    @ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p)
    def counts(args, stream):
        made.append(args)
        return 0

    entry(counts)
    call = getattr(fast, name)
    assert call(*good) is not None and len(made) == 1
    served = []
    for i, x in enumerate(good):
        for what, bad in worse(x).items():
            args = list(good)
            args[i] = bad
            before = len(made)
            if call(*args) is not None or len(made) != before:
                served.append((i, what))
    assert set(served) == ALLOWED[name]
