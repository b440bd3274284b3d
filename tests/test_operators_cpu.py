"""The training operators without a GPU: what they refuse, the size helpers,
and the pins of the tests' own restatements."""
import math

import numpy as np
import pytest

from tests import ops_ref as R


@pytest.fixture(scope="module")
def z():
    import __graft_entry__
    __graft_entry__._library_builder().build()
    import zero_sharded_optimizer_step_gb300 as z
    return z


def refused(z, code, fn, *args):
    with pytest.raises(z.ZeroError) as ei:
        fn(*args)
    assert ei.value.code == code, str(ei.value)
    assert z.zero_last_error()


A, B, C, D = 1 << 20, 2 << 20, 3 << 20, 4 << 20     # addresses; refused before any use


def edit(args, i, v):
    out = list(args)
    out[i] = v
    return out


def test_embed_refusals(z):
    ok = [A, z.ZERO_BF16, 100, 64, 64, B, 8, 10, -1, 1.0, C, 64, None, 0]
    for i, v in [(0, None), (1, 7), (2, -1), (3, -1), (3, 65), (4, 63), (5, None), (6, 2),
                 (6, 16), (7, -1), (7, 1 << 31), (9, math.inf), (9, math.nan), (10, None),
                 (11, 63), (4, 1 << 62)]:
        refused(z, z.ZERO_EINVAL, z.zero_embed, *edit(ok, i, v))
    for i, v in [(0, A + 1), (5, B + 4), (10, C + 1), (12, D + 4)]:
        refused(z, z.ZERO_EALIGN, z.zero_embed, *edit(ok, i, v))
    # nothing to do: nothing launched, on any machine
    z.zero_embed(None, z.ZERO_F32, 0, 64, 64, None, 4, 0, -1, 1.0, None, 64, None, 0)
    z.zero_embed(None, z.ZERO_F32, 5, 0, 0, B, 4, 9, -1, 1.0, None, 0, None, 0)


def test_embed_grad_refusals(z):
    need = z.zero_embed_grad_workspace(100, 64, 10)
    ok = [A, z.ZERO_BF16, 64, B, 8, 10, -1, 1.0, C, z.ZERO_F32, 100, 64, 64, False, D, need, 0]
    for i, v in [(0, None), (1, 3), (2, 63), (3, None), (4, 1), (5, -1), (5, 1 << 31),
                 (7, math.nan), (8, None), (9, -1), (10, -1), (11, -1), (12, 63), (14, None),
                 (15, need - 1), (15, 0)]:
        refused(z, z.ZERO_EINVAL, z.zero_embed_grad, *edit(ok, i, v))
    for i, v in [(0, A + 1), (3, B + 4), (8, C + 2), (14, D + 8)]:
        refused(z, z.ZERO_EALIGN, z.zero_embed_grad, *edit(ok, i, v))
    for bad in [(-1, 64, 10), (100, -1, 10), (100, 64, -1), (100, 64, 1 << 31)]:
        assert z.zero_embed_grad_workspace(*bad) == -1
    # every token, row and column more needs no less
    sizes = [z.zero_embed_grad_workspace(1000, 700, n) for n in (0, 1, 8, 9, 8192, 8193, 200000)]
    assert sizes[0] > 0 and sizes == sorted(sizes)
    z.zero_embed_grad(None, z.ZERO_F32, 64, None, 4, 0, -1, 1.0, None, z.ZERO_F32, 0, 64, 64,
                      False, None, 0, 0)
    z.zero_embed_grad(None, z.ZERO_F32, 64, None, 4, 0, -1, 1.0, C, z.ZERO_F32, 9, 64, 64,
                      True, None, 0, 0)


def test_dropout_refusals(z):
    ok = [A, None, B, z.ZERO_F16, 100, 0.1, 1, 2, 0, 0]
    for i, v in [(0, None), (2, None), (3, 9), (4, -1), (5, -0.1), (5, 1.1), (5, math.nan),
                 (8, -4), (8, 2)]:
        refused(z, z.ZERO_EINVAL, z.zero_dropout, *edit(ok, i, v))
    for i, v in [(0, A + 1), (1, C + 1), (2, B + 1)]:
        refused(z, z.ZERO_EALIGN, z.zero_dropout, *edit(ok, i, v))
    z.zero_dropout(None, None, None, z.ZERO_F32, 0, 0.5, 1, 2, 0, 0)


def test_mx4_refusals(z):
    ok = [A, z.ZERO_BF16, 10, 100, 100, B, C, 0]
    for i, v in [(0, None), (1, 4), (2, -1), (3, 1 << 31), (4, 99)]:
        refused(z, z.ZERO_EINVAL, z.zero_mx4_quantize, *edit(ok, i, v))
    refused(z, z.ZERO_EINVAL, z.zero_mx4_quantize, *edit(edit(ok, 5, None), 6, None))
    for i, v in [(0, A + 1), (5, B + 8), (6, C + 4)]:
        refused(z, z.ZERO_EALIGN, z.zero_mx4_quantize, *edit(ok, i, v))
    ok = [B, 10, 100, A, z.ZERO_F32, 100, 0]
    for i, v in [(0, None), (1, -1), (2, -1), (3, None), (4, 5), (5, 99)]:
        refused(z, z.ZERO_EINVAL, z.zero_mx4_dequantize, *edit(ok, i, v))
    for i, v in [(0, B + 8), (3, A + 2)]:
        refused(z, z.ZERO_EALIGN, z.zero_mx4_dequantize, *edit(ok, i, v))
    ok = [A, 10, B, 20, 100, 1.0, False, C, z.ZERO_F32, 20, 0]
    for i, v in [(0, None), (1, -1), (2, None), (3, -1), (4, -1), (5, math.inf), (7, None),
                 (8, 8), (9, 19)]:
        refused(z, z.ZERO_EINVAL, z.zero_mx4_matmul, *edit(ok, i, v))
    for i, v in [(0, A + 8), (2, B + 1), (7, C + 2)]:
        refused(z, z.ZERO_EALIGN, z.zero_mx4_matmul, *edit(ok, i, v))
    assert z.zero_mx4_bytes(-1, 5) == -1 and z.zero_mx4_bytes(5, 1 << 31) == -1
    for r, c, records in [(0, 5, 0), (1, 1, 1), (128, 256, 1), (129, 256, 2), (128, 257, 2),
                          (1000, 1000, 32)]:
        assert z.zero_mx4_bytes(r, c) == records * 17408
    assert z.zero_mx4_bytes((1 << 31) - 2, (1 << 31) - 2) == (1 << 24) * (1 << 23) * 17408


def test_philox_restatement_pins():
    """The known answers published with the generator (Random123)."""
    kat = [((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
           ((0xffffffff,) * 4, (0xffffffff,) * 2,
            (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
           ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
            (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1))]
    for c, k, want in kat:
        assert tuple(int(v) for v in R.philox([c], k)[0]) == want


def test_quantize_restatement_pins():
    """Hand-worked blocks: the largest magnitude sets the power of two, ties
    go to the even code, values past 6 to 6."""
    x = np.zeros((1, 32))
    x[0, :12] = [4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.9, -0.2, -6.0, 0.26]
    codes, scale = R.quantize(x)
    assert scale.tolist() == [[127]]                     # 2^(floor(log2 7.9) - 2) = 1
    assert R.values(codes, scale)[0, :12].tolist() == [4, 0, 1, 1, 2, 2, 4, 4, 6, 0, -6, 0.5]
    codes, scale = R.quantize(np.full((1, 3), 2.0 ** -140))
    assert scale.tolist() == [[0]] and R.values(codes, scale).tolist() == [[0, 0, 0]]
    x[0, 3] = np.inf
    assert R.quantize(x)[1].tolist() == [[255]]


def test_layers_refuse_what_is_not_on_a_gpu(z):
    import torch
    t, tok = torch.zeros(4, 8), torch.zeros(3, dtype=torch.int64)
    for bad in (lambda: z.embed(t, tok), lambda: z.embed_grad(t, tok, t),
                lambda: z.dropout(t, 0.5, 1, 2), lambda: z.mx4_quantize(t),
                lambda: z.Mx4Linear(t)):
        with pytest.raises(ValueError):
            bad()


def test_calls_convert_or_refuse_their_arguments(z):
    """The compiled marshalling: what is no pointer, whole number or number
    raises, and nothing is called; what converts reaches the library's checks."""
    from zero_sharded_optimizer_step_gb300 import _calls

    class Tensor:
        def __init__(self, at):
            self.at = at

        def data_ptr(self):
            return self.at

    class Broken:
        def data_ptr(self):
            raise KeyError("broken")

    ok = [A, None, B, z.ZERO_F32, 0, 0.1, 3, 4, 0, 5]     # no elements: nothing is launched
    z.zero_dropout(*ok)
    z.zero_dropout(*edit(ok, 0, Tensor(A)))
    z.zero_dropout(*edit(ok, 4, np.int64(0)))
    z.zero_dropout(*edit(ok, 5, 0))
    z.zero_dropout(*edit(ok, 6, (1 << 64) - 1))
    z.zero_dropout(*edit(ok, 6, -1))                      # the seed's 64 bits
    for i, v, error in [(0, "x", AttributeError), (0, Broken(), KeyError), (0, -1, OverflowError),
                        (2, Tensor("x"), TypeError), (3, 1 << 31, OverflowError),
                        (3, 0.5, TypeError), (4, 1 << 63, OverflowError), (4, None, TypeError),
                        (5, "x", TypeError), (6, 0.5, TypeError), (8, 1.0, TypeError)]:
        with pytest.raises(error):
            z.zero_dropout(*edit(ok, i, v))
    refused(z, z.ZERO_EINVAL, z.zero_dropout, *edit(ok, 0, Tensor(0))[:4], 4, *ok[5:])
    for name, n in [("embed", 14), ("embed_grad", 17), ("dropout", 10), ("quantize", 8),
                    ("dequantize", 7), ("matmul", 11), ("bind", 6)]:
        for count in (0, n - 1, n + 1):
            with pytest.raises(TypeError):
                getattr(_calls, name)(*[0] * count)
    with pytest.raises(TypeError):
        z.zero_dropout(*ok[:4])


def test_calls_pass_every_argument_in_its_place(tmp_path):
    """A second copy of the module, loaded from its own file and bound to callbacks
    that write down what they are given."""
    import ctypes as c
    import importlib.util
    import shutil

    import __graft_entry__
    path = str(tmp_path / "_calls.so")
    shutil.copy(__graft_entry__._library_builder().build_calls(), path)
    spec = importlib.util.spec_from_file_location("_calls", path)
    calls = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(calls)
    with pytest.raises(RuntimeError):
        calls.matmul(*[0] * 11)
    p, i, l, f, d, u = c.c_void_p, c.c_int32, c.c_int64, c.c_float, c.c_double, c.c_uint64
    signatures = {
        "embed": [p, i, l, l, l, p, i, l, l, f, p, l, p, p],
        "embed_grad": [p, i, l, p, i, l, l, f, p, i, l, l, l, i, p, l, p],
        "dropout": [p, p, p, i, l, d, u, u, l, p],
        "quantize": [p, i, l, l, l, p, p, p],
        "dequantize": [p, l, l, p, i, l, p],
        "matmul": [p, l, p, l, l, f, i, p, i, l, p]}
    seen, kept = [], []
    for types in signatures.values():
        kept.append(c.CFUNCTYPE(c.c_int, *types)(lambda *a: seen.append(a) or len(a)))
    calls.bind(*(c.cast(k, p).value for k in kept))
    big = {p: 1 << 63, l: -(1 << 62), i: -(1 << 30), f: 0.5, d: 1 / 3, u: (1 << 64) - 9}
    truth = {"embed_grad": 13, "matmul": 6}
    for name, types in signatures.items():
        given = [big[t] + k if t not in (f, d) else big[t] + k for k, t in enumerate(types)]
        if name in truth:
            given[truth[name]] = True
        assert getattr(calls, name)(*given) == len(types)
        assert list(seen.pop()) == given
