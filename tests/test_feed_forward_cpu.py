"""The norm, the 16-bit products, the gated block and the rows kept in 8 bits
without a GPU: what they refuse, their size helpers, how their arguments pass, and
the pins of the tests' own restatements."""
import ctypes as c
import math

import numpy as np
import pytest
import torch

from tests import ff_ref as F


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


def edit(args, i, v):
    out = list(args)
    out[i] = v
    return out


A, B, C, D, E, G, H, W = ((k + 1) << 20 for k in range(8))   # addresses; refused before any use
BIG = 1 << 31


def test_pack8_refusals_and_sizes(z):
    ok = [A, z.ZERO_BF16, 10, 100, 100, B, 0]
    for i, v in [(0, None), (1, 4), (2, -1), (3, BIG), (4, 99), (5, None)]:
        refused(z, z.ZERO_EINVAL, z.zero_pack8, *edit(ok, i, v))
    for i, v in [(0, A + 1), (5, B + 8)]:
        refused(z, z.ZERO_EALIGN, z.zero_pack8, *edit(ok, i, v))
    ok = [B, 10, 100, A, z.ZERO_F32, 100, 0]
    for i, v in [(0, None), (1, -1), (2, -1), (3, None), (4, 5), (5, 99)]:
        refused(z, z.ZERO_EINVAL, z.zero_unpack8, *edit(ok, i, v))
    for i, v in [(0, B + 8), (3, A + 2)]:
        refused(z, z.ZERO_EALIGN, z.zero_unpack8, *edit(ok, i, v))
    for r, k, want in [(0, 5, 0), (1, 1, 33), (1, 32, 33), (3, 33, 198), (1000, 1601, 1000 * 1683)]:
        assert z.zero_pack8_bytes(r, k) == want
    assert z.zero_pack8_bytes(-1, 5) == -1 and z.zero_pack8_bytes(5, BIG) == -1
    z.zero_pack8(None, z.ZERO_F32, 0, 64, 64, None, 0)          # nothing to do, on any machine
    z.zero_unpack8(None, 5, 0, C, z.ZERO_F32, 0, 0)


def test_norm_refusals(z):
    #     x  xs  res rs  w  dtype       rows dim eps  sum ss  y  ys  q    rstd stream
    ok = [A, 64, B, 64, C, z.ZERO_BF16, 10, 64, 1e-5, D, 64, E, 64, None, G, 0]
    for i, v in [(0, None), (1, 63), (3, 63), (4, None), (5, 3), (6, -1), (7, -1), (7, 65),
                 (8, -1.0), (8, math.nan), (8, math.inf), (10, 63), (11, None), (12, 63)]:
        refused(z, z.ZERO_EINVAL, z.zero_rms_norm, *edit(ok, i, v))
    for i, v in [(0, A + 1), (2, B + 1), (4, C + 1), (9, D + 1), (11, E + 1), (13, H + 8),
                 (14, G + 2)]:
        refused(z, z.ZERO_EALIGN, z.zero_rms_norm, *edit(ok, i, v))
    z.zero_rms_norm(*edit(edit(ok, 0, None), 6, 0))
    need = z.zero_rms_norm_grad_workspace(10, 64)
    #     dy ds      s      w  rstd dtype         rows dim dx    dw  grad        acc    ws need st
    ok = [A, 64, B, 64, C, 64, D, E, z.ZERO_BF16, 10, 64, G, 64, H, z.ZERO_F32, False, W, need, 0]
    for i, v in [(0, None), (1, 63), (3, 63), (4, None), (5, 63), (6, None), (7, None), (8, 9),
                 (9, -1), (10, -1), (11, None), (12, 63), (14, 7), (16, None), (17, need - 1)]:
        refused(z, z.ZERO_EINVAL, z.zero_rms_norm_grad, *edit(ok, i, v))
    for i, v in [(0, A + 1), (2, B + 1), (4, C + 1), (6, D + 1), (7, E + 2), (11, G + 1),
                 (13, H + 2), (16, W + 8)]:
        refused(z, z.ZERO_EALIGN, z.zero_rms_norm_grad, *edit(ok, i, v))
    z.zero_rms_norm_grad(*edit(edit(ok, 9, 0), 15, True))         # no rows: nothing to add
    assert z.zero_rms_norm_grad_workspace(-1, 4) == -1
    assert z.zero_rms_norm_grad_workspace(4, BIG) == -1
    for dim in (1, 700, 768, 1000, 4096, 8192, 8193, 20000):
        sizes = [z.zero_rms_norm_grad_workspace(n, dim) for n in (0, 1, 9, 100, 10 ** 6, 2 ** 31 - 2)]
        assert sizes == sorted(sizes) and sizes[1] >= 4 * dim


def test_product_refusals(z):
    #     a  t      as  b  t      bs  a2    as  b2    bs  dtype         m   n   k
    ok = [A, False, 64, B, False, 64, None, 64, None, 64, z.ZERO_BF16, 100, 40, 64,
          C, 4, D, 40, E, 40, None, G, z.ZERO_BF16, 40, False, None, 0, 0]
    for i, v in [(0, None), (2, 63), (3, None), (5, 63), (10, z.ZERO_F32), (10, 5), (11, -1),
                 (12, -1), (13, -1), (11, BIG), (13, 65), (15, 5), (15, -1), (17, 39), (19, 39),
                 (20, H), (21, None), (22, z.ZERO_F16), (23, 39), (24, True), (6, H), (8, H)]:
        refused(z, z.ZERO_EINVAL, z.zero_matmul, *edit(ok, i, v))
    for i, v in [(0, A + 1), (3, B + 1), (14, C + 1), (16, D + 1), (18, E + 1), (21, G + 1)]:
        refused(z, z.ZERO_EALIGN, z.zero_matmul, *edit(ok, i, v))
    refused(z, z.ZERO_EALIGN, z.zero_matmul, *edit(edit(ok, 18, None), 20, H + 8))
    # rows of the transposes are as long as the result's sides
    refused(z, z.ZERO_EINVAL, z.zero_matmul, *edit(edit(ok, 1, True), 2, 99))
    refused(z, z.ZERO_EINVAL, z.zero_matmul, *edit(edit(ok, 4, True), 5, 39))
    pairs = edit(edit(ok, 6, H), 8, W)
    for i, v in [(7, 63), (9, 63), (6, None)]:
        refused(z, z.ZERO_EINVAL, z.zero_matmul, *edit(pairs, i, v))
    # rows off the boundaries need the workspace
    off = edit(edit(ok, 2, 65), 0, A + 2)
    need = z.zero_matmul_workspace(*off[:10], 100, 40, 64)
    assert need >= 100 * 64 * 2
    for ws, size, code in [(None, need, z.ZERO_EINVAL), (H, need - 1, z.ZERO_EINVAL),
                           (H + 8, need, z.ZERO_EALIGN)]:
        refused(z, code, z.zero_matmul, *off[:25], ws, size, 0)
    z.zero_matmul(*edit(ok, 11, 0))                               # nothing to do
    z.zero_matmul(*edit(edit(ok, 12, 0), 3, None))


def test_product_workspace(z):
    def need(a, ta, sa, b, tb, sb, m, n, k, a2=None, b2=None):
        return z.zero_matmul_workspace(a, ta, sa, b, tb, sb, a2, sa, b2, sb, m, n, k)

    assert need(A, False, 64, B, False, 64, 100, 40, 64) == 0
    assert need(A, False, 65, B, False, 64, 100, 40, 65) >= 100 * 72 * 2
    assert need(A, True, 100, B, False, 64, 100, 40, 64) >= 64 * 104 * 2
    assert need(A, True, 104, B, True, 40, 100, 40, 64) == 0
    assert need(A + 8, False, 64, B + 2, False, 64, 100, 40, 64) >= 140 * 64 * 2
    one = need(A, False, 65, B, False, 72, 100, 40, 65)
    assert need(A, False, 65, B, False, 72, 100, 40, 65, C, D) == 2 * one
    assert need(A, False, 65, B, False, 65, 1, 40, 65) == 0       # one row is read as it lies
    assert need(A, False, 64, B, False, 64, -1, 40, 64) == -1
    assert need(A, False, 64, B, False, 64, 5, 40, BIG) == -1
    assert z.zero_gated_workspace(A, 64, B, 64, C, 64, 100, 40, 64) == 0
    assert z.zero_gated_workspace(A, 64, B, 65, C, 65, 100, 40, 64) >= 2 * 40 * 64 * 2
    assert z.zero_gated_workspace(A, 64, B, 64, C, 64, 100, -1, 64) == -1


def test_gated_refusals(z):
    #     x  xs  wg gs  wu us  dtype         m   n   k   act gate up ks  gq    uq   h  hs ws    need st
    ok = [A, 64, B, 64, C, 64, z.ZERO_F16, 100, 40, 64, 4, D, E, 40, None, None, G, 40, None, 0, 0]
    for i, v in [(0, None), (1, 63), (2, None), (3, 63), (4, None), (5, 63), (6, z.ZERO_F32),
                 (7, -1), (8, -1), (9, 65), (10, 9), (11, None), (12, None), (13, 39), (14, H),
                 (16, None), (17, 39)]:
        refused(z, z.ZERO_EINVAL, z.zero_gated, *edit(ok, i, v))
    refused(z, z.ZERO_EINVAL, z.zero_gated, *edit(edit(ok, 14, H), 15, W))      # both kinds
    for i, v in [(0, A + 1), (2, B + 1), (4, C + 1), (11, D + 1), (12, E + 1), (16, G + 1)]:
        refused(z, z.ZERO_EALIGN, z.zero_gated, *edit(ok, i, v))
    off = edit(ok, 0, A + 2)
    refused(z, z.ZERO_EINVAL, z.zero_gated, *off)                 # the workspace is missing
    z.zero_gated(*edit(ok, 7, 0))
    #     dh hs  g  u  ks  gq    uq    act dtype        rows cols dg du gs  h  hs st
    ok = [A, 64, B, C, 64, None, None, 4, z.ZERO_BF16, 10, 64, D, E, 64, G, 64, 0]
    for i, v in [(0, None), (1, 63), (2, None), (3, None), (4, 63), (5, H), (7, 5), (8, 7),
                 (9, -1), (10, BIG), (11, None), (12, None), (13, 63), (15, 63)]:
        refused(z, z.ZERO_EINVAL, z.zero_gated_grad, *edit(ok, i, v))
    refused(z, z.ZERO_EINVAL, z.zero_gated_grad, *edit(edit(ok, 2, None), 3, None))
    for i, v in [(0, A + 1), (2, B + 1), (3, C + 1), (11, D + 1), (12, E + 1), (14, G + 1)]:
        refused(z, z.ZERO_EALIGN, z.zero_gated_grad, *edit(ok, i, v))
    z.zero_gated_grad(*edit(ok, 9, 0))


def test_activation_gradient_refusals(z):
    need = z.zero_activation_grad_workspace(10, 64)
    #     dy ys  z  zs  q     act dtype       rows cols dz ds  db bdtype       acc    ws need st
    ok = [A, 64, B, 64, None, 2, z.ZERO_F16, 10, 64, C, 64, D, z.ZERO_F32, False, W, need, 0]
    for i, v in [(0, None), (1, 63), (2, None), (3, 63), (4, H), (5, -1), (6, 3), (7, -1),
                 (8, -1), (10, 63), (12, 4), (14, None), (15, need - 1)]:
        refused(z, z.ZERO_EINVAL, z.zero_activation_grad, *edit(ok, i, v))
    refused(z, z.ZERO_EINVAL, z.zero_activation_grad, *edit(edit(ok, 9, None), 11, None))
    for i, v in [(0, A + 1), (2, B + 1), (9, C + 1), (11, D + 2), (14, W + 8)]:
        refused(z, z.ZERO_EALIGN, z.zero_activation_grad, *edit(ok, i, v))
    z.zero_activation_grad(*edit(edit(ok, 7, 0), 13, True))
    assert z.zero_activation_grad_workspace(-1, 4) == -1
    assert z.zero_activation_grad_workspace(4, BIG) == -1


def test_layers_refuse_what_is_not_on_a_gpu(z):
    t, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.ones(8, dtype=torch.bfloat16)
    for bad in (lambda: z.pack8(t), lambda: z.rms_norm(t, w), lambda: z.linear(t, t),
                lambda: z.gated(t, t, t), lambda: z.matmul(t, t),
                lambda: z.linear(t, w), lambda: z.gated(t, w, w)):
        with pytest.raises(ValueError):
            bad()


SIGNATURES = {
    "pack8": "pilllpp", "unpack8": "pllpilp", "rms_norm": "plplpillfplplppp",
    "rms_norm_grad": "plplplppillplpitplp", "product_workspace": "ptlptlplpllll",
    "product": "ptlptlplplilllpiplplppiltplp", "gated_workspace": "plplpllll",
    "gated": "plplplilllipplppplplp",
    "activation_grad": "plplpiillplpitplp", "gated_grad": "plpplppiillpplplp",
    "pack8_bytes": "ll", "norm_workspace": "ll", "activation_workspace": "ll"}
SIZES = ("product_workspace", "gated_workspace", "pack8_bytes", "norm_workspace",
         "activation_workspace")


def test_calls_pass_every_argument_in_its_place(tmp_path):
    """A second copy of the module, loaded from its own file and bound to callbacks
    that write down what they are given."""
    import importlib.util
    import shutil

    import __graft_entry__
    path = str(tmp_path / "_calls.so")
    shutil.copy(__graft_entry__._library_builder().build_calls(), path)
    spec = importlib.util.spec_from_file_location("_calls", path)
    calls = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(calls)
    with pytest.raises(RuntimeError):
        calls.pack8(*[0] * 7)
    kind = {"p": c.c_void_p, "i": c.c_int32, "t": c.c_int32, "l": c.c_int64, "f": c.c_float}
    big = {"p": 1 << 62, "l": -(1 << 61), "i": -(1 << 29), "f": 0.5}
    seen, kept = [], []
    for name, types in SIGNATURES.items():
        back = c.c_int64 if name in SIZES else c.c_int
        kept.append(c.CFUNCTYPE(back, *(kind[t] for t in types))(
            lambda *a: seen.append(a) or len(a)))
    calls.bind_layers(*(c.cast(k, c.c_void_p).value for k in kept))
    for name, types in SIGNATURES.items():
        given = [k % 2 == 0 if t == "t" else big[t] + k for k, t in enumerate(types)]
        assert getattr(calls, name)(*given) == len(types)
        assert list(seen.pop()) == [int(v) if t == "t" else v for v, t in zip(given, types)]
        for count in (0, len(types) - 1, len(types) + 1):
            with pytest.raises(TypeError):
                getattr(calls, name)(*[0] * count)
        for k, t in enumerate(types):
            with pytest.raises((AttributeError, TypeError)):
                getattr(calls, name)(*edit(given, k, "x" if t != "t" else Broken()))
    assert not seen
    for count in (0, 12, 14):
        with pytest.raises(TypeError):
            calls.bind_layers(*[0] * count)


class Broken:
    def __bool__(self):
        raise TypeError("broken")


def test_pack_restatement_pins():
    """Hand-worked blocks: the largest magnitude sets the smallest scale that
    holds it below 448, ties go to the even code, subnormal codes are spaced 2^-9."""
    x = torch.zeros(1, 32, dtype=torch.float64)
    x[0, :9] = torch.tensor([448.0, 17.0, 19.0, -17.0, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -9, 0.1,
                             1.0625])
    v, e = F.pack(x)
    assert e.tolist() == [[127]]
    assert v[0, :9].tolist() == [448, 16, 20, -16, 0, 2 * 2.0 ** -9, 2.0 ** -9, 0.1015625, 1]
    x[0, 0] = 448.5                                   # 2^1: everything is halved first
    v, e = F.pack(x)
    assert e.tolist() == [[128]] and v[0, 0] == 448 and v[0, 1] == 16 and v[0, 2] == 20
    v, e = F.pack(torch.full((1, 3), 2.0 ** -140, dtype=torch.float64))
    assert e.tolist() == [[0]] and v.tolist() == [[0, 0, 0]]
    x[0, 3] = math.inf
    v, e = F.pack(x)
    assert e.tolist() == [[255]] and torch.isnan(v).all()
    assert F.rounded(torch.tensor([65536.0]).double(), torch.float16).item() == 65504


def test_activation_restatement_pins():
    """Known values, and slopes against differences."""
    v = torch.tensor([-2.0, -0.5, 0.0, 0.5, 3.0], dtype=torch.float64)
    want = {F.RELU: [0, 0, 0, 0.5, 3], F.NONE: v.tolist(),
            F.SILU: [-2 / (1 + math.e ** 2), -0.5 / (1 + math.e ** 0.5), 0,
                     0.5 / (1 + math.e ** -0.5), 3 / (1 + math.e ** -3)],
            F.GELU: [x * 0.5 * (1 + math.erf(x / math.sqrt(2))) for x in v.tolist()],
            F.GELU_TANH: [0.5 * x * (1 + math.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)))
                          for x in v.tolist()]}
    h = 1e-6
    for kind, w in want.items():
        y, slope = F.activation(v, kind)
        assert np.allclose(y, w, rtol=1e-14, atol=1e-15)
        d = (F.activation(v + h, kind)[0] - F.activation(v - h, kind)[0]) / (2 * h)
        keep = v != 0 if kind == F.RELU else v == v
        assert np.allclose(slope[keep], d[keep], atol=1e-9)
