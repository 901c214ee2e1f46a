"""Linear attention over sequences and rotary positions without a GPU: the oracle against differences, arguments and sizes."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import linear_seq as ref
from speculative_decoding_linear_gb300 import build as gbuild
from speculative_decoding_linear_gb300 import gdnspec
from test_seq_oracle import BAD, SHAPE, backward_args, far, forward_args, step_args

NO_GPU = (gdnspec.ERR_CUDA, gdnspec.ERR_DEVICE)
without_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="a valid call would launch on made-up addresses")


@pytest.fixture(scope="module")
def L():
    gbuild.build()
    return gdnspec.lib()


def problem(lengths=(3, 0, 36), H=4, Hk=2, dk=6, dv=5, seed=0):
    rng = np.random.default_rng(seed)
    t, n = sum(lengths), len(lengths)
    x = dict(q=rng.standard_normal((t, Hk, dk)), k=rng.standard_normal((t, Hk, dk)), v=rng.standard_normal((t, H, dv)),
             log_alpha=-rng.uniform(0.01, 1.0, (t, H)), beta=rng.uniform(0.1, 1.0, (t, H)), S0=rng.standard_normal((n, H, dv, dk)))
    return x, lengths, rng.standard_normal((t, H, dv)), rng.standard_normal((n, H, dv, dk))


@pytest.mark.parametrize("name", ["q", "k", "v", "log_alpha", "beta", "S0"])
def test_gradients_against_differences(name):
    x, lengths, do, dS = problem()
    g = ref.backward(**x, lengths=lengths, dout=do, dS_T=dS)[name]
    u = np.random.default_rng(1).standard_normal(g.shape)

    def loss(e):
        o, S = ref.forward(**dict(x, **{name: x[name] + e * u}), lengths=lengths)
        return (o * do).sum() + (S * dS).sum()

    e = 1e-6
    # third derivatives of order one: the central difference is off by e^2, its sums by 1e-16 / e of the loss
    assert abs((loss(e) - loss(-e)) / (2 * e) - (g * u).sum()) < 1e-6 * max(1.0, abs((g * u).sum()))


def test_segments_give_the_same_states():
    """What the kernels rest on: a sequence in pieces, each from the state before it."""
    x, lengths, _, _ = problem(lengths=(40,))
    whole, S = ref.forward(**x, lengths=lengths)
    state, at = x["S0"], 0
    for n in (1, 17, 22):
        piece = {m: y[at:at + n] for m, y in x.items() if m != "S0"}
        o, state = ref.forward(**piece, S0=state, lengths=(n,))
        assert np.allclose(o, whole[at:at + n], rtol=1e-12, atol=1e-12)
        at += n
    assert np.allclose(state, S, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_depends_on_differences_and_inverts(interleaved):
    rng = np.random.default_rng(2)
    f = ref.rotary_frequencies(16, 10000.0, 1.0, 0.0, 1.0, 32.0)
    q, k = rng.standard_normal((1, 1, 24)), rng.standard_normal((1, 1, 24))
    at = lambda x, p: ref.rotary(x, np.array([p]), f, interleaved=interleaved)  # noqa: E731
    assert np.allclose((at(q, 7) * at(k, 3)).sum(), (at(q, 104) * at(k, 100)).sum())
    y = at(q, 123456)
    assert np.allclose(ref.rotary(y, np.array([123456]), f, interleaved=interleaved, inverse=True), q)
    assert (y[..., 16:] == q[..., 16:]).all()
    # the inverse is the transpose: <R x, y> = <x, R^T y>
    assert np.allclose((y * k).sum(), (q * ref.rotary(k, np.array([123456]), f, interleaved=interleaved, inverse=True)).sum())


def types_of(bad):
    """Both types, but where the refusal depends on it (260 elements are whole 16 bytes in fp32)."""
    return (bad["dtype"],) if "dtype" in bad else (0,) if bad.get("ldk") == 4 * 64 + 4 else (0, 1)


@pytest.mark.parametrize("bad", BAD + [dict(out=None), dict(S0=far(5) + 4), dict(out=far(2)), dict(S_T=far(5) + 256), dict(rec=far(7)),
                                       dict(ws=far(0)), dict(rec=far(9) + 8), dict(ws=far(10) + 4)])
def test_forward_refuses(L, bad):
    for dtype in types_of(bad):
        assert L.gdn_linear_seq_forward(*forward_args(**dict(bad, dtype=dtype))) == gdnspec.ERR_ARG


@pytest.mark.parametrize("bad", BAD + [dict(dout=None), dict(rec=None), dict(dq=None), dict(dkk=far(9)), dict(dvv=far(6)), dict(dla=None),
                                       dict(dbeta=far(12)), dict(dS0=far(7) + 256), dict(ws=far(8)), dict(rec=far(8) + 4)])
def test_backward_refuses(L, bad):
    for dtype in types_of(bad):
        assert L.gdn_linear_seq_backward(*backward_args(**dict(bad, dtype=dtype))) == gdnspec.ERR_ARG


@pytest.mark.parametrize("Hk,dk", [(1 << 23, 256), (1 << 24, 256), (1 << 24, 128)])
def test_rows_wider_than_an_int_counts(L, Hk, dk):
    shape = dict(nseq=1, total=1, H=Hk, Hk=Hk, dk=dk, dv=16, ldq=8, ldk=8, ldv=16 * Hk, off=None, dtype=1)
    assert L.gdn_linear_seq_forward(*forward_args(**shape)) == gdnspec.ERR_ARG
    assert L.gdn_linear_seq_backward(*backward_args(**shape)) == gdnspec.ERR_ARG


@pytest.mark.parametrize("bad", [dict(B=0), dict(slots=0), dict(H=0), dict(Hk=3), dict(dk=8), dict(dv=20), dict(dtype=-1), dict(q=None),
                                 dict(S=None), dict(S=far(5) + 4), dict(out=far(5)), dict(out=far(2)), dict(index=None, slots=3),
                                 dict(index=far(6) + 2)])
def test_step_refuses(L, bad):
    assert L.gdn_linear_seq_step(*step_args(**bad)) == gdnspec.ERR_ARG


def rotary_args(**kw):
    a = dict(q=far(0), ldq=512, k=far(1), ldk=128, dtype=0, pos=far(2), freq=far(3), scale=1.0, qo=far(4), ldqo=512, ko=far(5),
             ldko=128, total=9, H=8, Hk=2, d=64, rot=32, inter=0, inv=0)
    a.update(kw)
    return [*a.values(), None]


@pytest.mark.parametrize("bad", [
    dict(total=-1), dict(H=0), dict(Hk=-1), dict(d=24), dict(d=272), dict(rot=0), dict(rot=66), dict(rot=31), dict(dtype=2), dict(q=None),
    dict(k=None), dict(ko=None), dict(Hk=0), dict(pos=None), dict(freq=None), dict(pos=far(2) + 2), dict(freq=far(3) + 1), dict(q=far(0) + 8),
    dict(qo=far(4) + 2), dict(ldq=511), dict(ldq=504), dict(ldk=120), dict(ldqo=516), dict(ldko=64), dict(inter=2), dict(inv=-1),
    dict(qo=far(1)), dict(ko=far(4)), dict(ko=far(0)), dict(qo=far(0), ldqo=520), dict(qo=far(0) + 16), dict(qo=far(2)), dict(ko=far(3)),
    dict(H=65534)])
def test_rotary_refuses(L, bad):
    assert L.gdn_rotary(*rotary_args(**bad)) == gdnspec.ERR_ARG


@without_gpu
def test_valid_calls_without_a_gpu_fail_loudly(L):
    for dtype in (0, 1):
        assert L.gdn_linear_seq_forward(*forward_args(dtype=dtype)) in NO_GPU
        assert L.gdn_linear_seq_forward(*forward_args(dtype=dtype, S_T=far(5))) in NO_GPU        # in place is allowed
        assert L.gdn_linear_seq_backward(*backward_args(dtype=dtype)) in NO_GPU
        assert L.gdn_linear_seq_backward(*backward_args(dtype=dtype, dS0=far(7))) in NO_GPU
        assert L.gdn_rotary(*rotary_args(dtype=dtype)) in NO_GPU
    assert L.gdn_linear_seq_step(*step_args()) in NO_GPU
    assert L.gdn_rotary(*rotary_args(qo=far(0), ko=far(1))) in NO_GPU                            # in place
    assert L.gdn_rotary(*rotary_args(k=None, ko=None, Hk=0)) in NO_GPU
    wide = dict(q=far(0), ldq=1024, k=far(0) + 1024, ldk=1024)                                   # columns of one projection
    assert L.gdn_rotary(*rotary_args(**wide, qo=far(0), ldqo=1024, ko=far(0) + 1024, ldko=1024)) in NO_GPU
    assert L.gdn_rotary(*rotary_args(**wide, qo=far(0) + 1280, ldqo=1024)) == gdnspec.ERR_ARG    # runs into the next row's q
    assert L.gdn_rotary(*rotary_args(total=0, q=None, k=None, qo=None, ko=None, pos=None)) == gdnspec.OK


def test_sizes(L):
    n = ctypes.c_size_t(0)
    for name in ("workspace", "forward_workspace", "record"):
        f = getattr(L, "gdn_linear_seq_%s_bytes" % name)
        assert f(1, 64, 8, 3, 64, 64, 0, ctypes.byref(n)) == gdnspec.ERR_ARG
        assert f(1, 64, 8, 4, 64, 64, 2, ctypes.byref(n)) == gdnspec.ERR_ARG
        assert f(1, 64, 8, 4, 64, 64, 0, None) == gdnspec.ERR_ARG
        for dtype in (0, 1):
            assert f(3, 0, 8, 8, 256, 256, dtype, ctypes.byref(n)) == 0 and n.value > 0
    dims = (3, 1000, 8, 8, 256, 256)
    for dtype in ("bf16", "f32"):
        assert 0 < gdnspec.gdn_linear_seq_forward_workspace_bytes(*dims, dtype) <= gdnspec.gdn_linear_seq_workspace_bytes(*dims, dtype)
    # fp32: a state for each 64 tokens
    assert gdnspec.gdn_linear_seq_record_bytes(*dims, "f32") >= (1000 // 64 + 3) * 8 * 256 * 256 * 4


@pytest.mark.parametrize("rot,base,factor,original", [(64, 1e4, 1.0, 0.0), (64, 1e4, 8.0, 4096.0), (2, 500.0, 4.0, 0.0), (256, 1e6, 32.0, 8192.0)])
def test_frequencies(L, rot, base, factor, original):
    f = gdnspec.gdn_rotary_frequencies(rot, base, factor, original, device="cpu")
    r = ref.rotary_frequencies(rot, base, factor, original, 1.0, 32.0)
    assert f.dtype == torch.float32 and np.abs(f.double().numpy() / r - 1).max() <= 2.0 ** -24 + 1e-14
    if original == 0.0:
        assert np.allclose(f.double().numpy() * factor, base ** (-2.0 * np.arange(rot // 2) / rot), rtol=1e-7)


@pytest.mark.parametrize("bad", [dict(rot=0), dict(rot=3), dict(rot=258), dict(base=0.0), dict(base=float("nan")), dict(factor=0.0),
                                 dict(factor=float("inf")), dict(original=-1.0), dict(original=10.0, low=2.0, high=2.0)])
def test_frequencies_refuse(L, bad):
    with pytest.raises((gdnspec.GdnError, ValueError)):
        gdnspec.gdn_rotary_frequencies(**dict(dict(rot=64, base=1e4, factor=2.0, original=0.0, device="cpu"), **bad))


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    x, g, p, f = torch.zeros(4, 2, 16), torch.zeros(4, 2), torch.zeros(4, dtype=torch.int32), torch.zeros(8)
    with pytest.raises(ValueError):
        gdnspec.gdn_linear_seq_forward(x, x, x, g, g, None, x, None, torch.zeros(1 << 20, dtype=torch.uint8))
    with pytest.raises(ValueError):
        gdnspec.gdn_linear_seq_forward(x, x[:, :1], x, g, g, None, x, None, None)
    with pytest.raises(ValueError):
        gdnspec.gdn_linear_seq_step(x, x, x, g, g, torch.zeros(4, 2, 16, 16), x)
    with pytest.raises(ValueError):
        gdnspec.gdn_linear_seq_step(x, x, x, g, g[:1], torch.zeros(4, 2, 16, 16), x)
    for bad in (dict(p=p[:3]), dict(p=p.long()), dict(k=x[:3]), dict(k=None), dict(f=f.double()), dict(ko=x[:, :1]), dict()):
        a = dict(dict(q=x, k=x, p=p, f=f, qo=x, ko=x), **bad)
        with pytest.raises(ValueError):
            gdnspec.gdn_rotary(*a.values())
    assert SHAPE["H"] % SHAPE["Hk"] == 0
