"""The fp64 sequence and norm oracles against differences and the tree oracle, and the entry points' refusals (CPU)."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from oracle import seq
from speculative_decoding_linear_gb300 import build as gbuild
from speculative_decoding_linear_gb300 import gdnspec


def inputs(rng, lengths, H, Hk, dk, dv):
    total = sum(lengths)
    unit = lambda *s: (lambda x: x / np.linalg.norm(x, axis=-1, keepdims=True))(rng.standard_normal(s))  # noqa: E731
    return dict(q=unit(total, Hk, dk), k=unit(total, Hk, dk), v=rng.standard_normal((total, H, dv)),
                log_alpha=-np.logaddexp(0, rng.uniform(-4, 1, (total, H))), beta=rng.uniform(0.1, 0.9, (total, H)),
                S0=0.3 * rng.standard_normal((len(lengths), H, dv, dk)))


def test_forward_is_the_chain_oracle():
    rng = np.random.default_rng(0)
    x = inputs(rng, [7], 2, 2, 4, 3)
    out, S_T = seq.seq_forward(**x, lengths=[7])
    parent = np.arange(-1, 6, dtype=np.int32)[None]
    b = {m: x[m][None] for m in ("q", "k", "v")}
    args = dict(alpha=np.exp(x["log_alpha"])[None], beta=x["beta"][None], parent=parent, S0=x["S0"])
    oracle.build()
    o, _, _ = oracle.tree_verify(**b, **args)
    np.testing.assert_allclose(out[None], o, rtol=1e-12, atol=1e-12)
    S = oracle.commit(b["k"], b["v"], args["alpha"], args["beta"], parent, x["S0"], np.arange(7, dtype=np.int32)[None])
    np.testing.assert_allclose(S_T, S, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("H,Hk", [(2, 2), (4, 2)])
def test_backward_against_differences(H, Hk):
    rng = np.random.default_rng(1)
    lengths = [3, 0, 5]
    x = inputs(rng, lengths, H, Hk, 4, 3)
    dout, dS = rng.standard_normal(x["v"].shape), rng.standard_normal(x["S0"].shape)
    got = seq.seq_backward(**x, lengths=lengths, dout=dout, dS_T=dS)

    def loss(y):
        o, S = seq.seq_forward(**y, lengths=lengths)
        return (o * dout).sum() + (S * dS).sum()

    h = 1e-5
    for name in x:
        d = rng.standard_normal(x[name].shape)
        up, dn = (dict(x, **{name: x[name] + s * h * d}) for s in (1, -1))
        want = (loss(up) - loss(dn)) / (2 * h)
        assert abs((got[name] * d).sum() - want) <= 1e-7 * max(1.0, abs(want)), name


def test_norm_gradients_against_differences():
    rng = np.random.default_rng(2)
    o, z, w, dy = (rng.standard_normal(s) for s in ((5, 6), (5, 6), (6,), (5, 6)))
    got = seq.gated_norm_backward(o, z, w, dy, 1e-3)
    h = 1e-5
    for i, base in enumerate((o, z, w)):
        d = rng.standard_normal(base.shape)
        f = lambda s: (seq.gated_norm(*[a + s * h * d if j == i else a for j, a in enumerate((o, z, w))], 1e-3) * dy).sum()  # noqa: E731
        want = (f(1) - f(-1)) / (2 * h)
        assert abs((got[i] * d).sum() - want) <= 1e-7 * max(1.0, abs(want))
    x, zz, wp, g, w = (rng.standard_normal(s) for s in ((4, 8), (4, 8), (8,), (8,), (8,)))
    dh, dx2 = rng.standard_normal((4, 8)), rng.standard_normal((4, 8))
    x2, _ = seq.block_norm(x, zz, wp, g, w, 1e-3, 0.9)
    dx, dz, dwp, dg, dw = seq.block_norm_backward(x2, zz, wp, g, w, dh, dx2, 1e-3, 0.9)
    for i, grad in enumerate((dx, dz, dwp, dg, dw)):
        d = rng.standard_normal(grad.shape)

        def f(s):
            a = [b + s * h * d if j == i else b for j, b in enumerate((x, zz, wp, g, w))]
            u, hh = seq.block_norm(*a, 1e-3, 0.9)
            return (u * dx2).sum() + (hh * dh).sum()
        want = (f(1) - f(-1)) / (2 * h)
        assert abs((grad * d).sum() - want) <= 1e-7 * max(1.0, abs(want))


# ---------------------------------------------------------------------------
# refusals: host-side checks that return before any CUDA call
# ---------------------------------------------------------------------------
@pytest.fixture(scope="module")
def L():
    gbuild.build()
    return gdnspec.lib()


def far(i):
    return (i + 1) << 40          # addresses that nothing overlaps and nothing dereferences


SHAPE = dict(nseq=2, total=64, H=8, Hk=4, dk=64, dv=128)


def forward_args(**kw):
    s = dict(SHAPE, **{k: v for k, v in kw.items() if k in SHAPE})
    a = dict(q=far(0), ldq=s["Hk"] * s["dk"], k=far(1), ldk=s["Hk"] * s["dk"], v=far(2), ldv=s["H"] * s["dv"], dtype=0,
             la=far(3), beta=far(4), S0=far(5), off=far(6), out=far(7), S_T=far(8), rec=far(9), ws=far(10))
    a.update({k: v for k, v in kw.items() if k in a})
    return [*a.values(), *s.values(), None]


def backward_args(**kw):
    s = dict(SHAPE, **{k: v for k, v in kw.items() if k in SHAPE})
    a = dict(q=far(0), ldq=s["Hk"] * s["dk"], k=far(1), ldk=s["Hk"] * s["dk"], v=far(2), ldv=s["H"] * s["dv"], dtype=0,
             la=far(3), beta=far(4), off=far(5), dout=far(6), dS_T=far(7), rec=far(8), dq=far(9), dkk=far(10), dvv=far(11),
             dla=far(12), dbeta=far(13), dS0=far(14), ws=far(15))
    a.update({k: v for k, v in kw.items() if k in a})
    return [*a.values(), *s.values(), None]


BAD = [dict(nseq=0), dict(total=-1), dict(H=0), dict(Hk=0), dict(Hk=3), dict(dk=24), dict(dk=272), dict(dv=8), dict(dtype=2),
       dict(ldq=8), dict(ldk=4 * 64 + 4), dict(ldv=100), dict(q=None), dict(k=far(1) + 8), dict(v=None), dict(la=None), dict(la=far(3) + 2),
       dict(beta=None), dict(ws=None), dict(off=far(6) + 2), dict(off=None, total=63)]


@pytest.mark.parametrize("bad", BAD + [dict(out=None), dict(S0=far(5) + 4), dict(out=far(2)), dict(S_T=far(5) + 256),
                                       dict(rec=far(7)), dict(ws=far(0))])
def test_seq_forward_refuses(L, bad):
    assert L.gdn_seq_forward(*forward_args(**bad)) == gdnspec.ERR_ARG


@pytest.mark.parametrize("bad", BAD + [dict(dout=None), dict(rec=None), dict(dq=None), dict(dkk=far(9)), dict(dvv=far(6)),
                                       dict(dla=None), dict(dbeta=far(12)), dict(dS0=far(7) + 256), dict(ws=far(8))])
def test_seq_backward_refuses(L, bad):
    assert L.gdn_seq_backward(*backward_args(**bad)) == gdnspec.ERR_ARG


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU failure mode")
def test_valid_calls_without_a_gpu_fail_loudly(L):
    no_gpu = (gdnspec.ERR_CUDA, gdnspec.ERR_DEVICE)
    assert L.gdn_seq_forward(*forward_args()) in no_gpu
    assert L.gdn_seq_forward(*forward_args(S_T=far(5))) in no_gpu        # in place is allowed
    assert L.gdn_seq_backward(*backward_args()) in no_gpu
    assert L.gdn_seq_step(*step_args()) in no_gpu
    assert L.gdn_gated_norm(*gated_args()) in no_gpu
    assert L.gdn_block_norm(*block_args()) in no_gpu


def step_args(**kw):
    a = dict(q=far(0), k=far(1), v=far(2), dtype=0, la=far(3), beta=far(4), S=far(5), index=far(6), out=far(7), B=4, slots=6,
             H=8, Hk=2, dk=64, dv=128)
    a.update(kw)
    return [*a.values(), None]


@pytest.mark.parametrize("bad", [dict(B=0), dict(slots=0), dict(H=0), dict(Hk=3), dict(dk=8), dict(dv=20), dict(dtype=-1),
                                 dict(q=None), dict(S=None), dict(S=far(5) + 4), dict(out=far(5)), dict(out=far(2)),
                                 dict(index=None, slots=3), dict(index=far(6) + 2)])
def test_seq_step_refuses(L, bad):
    assert L.gdn_seq_step(*step_args(**bad)) == gdnspec.ERR_ARG


def gated_args(**kw):
    a = dict(o=far(0), ot=1, gate=far(1), w=far(2), out=far(3), dtype=0, rows=10, d=64, eps=1e-6)
    a.update(kw)
    return [*a.values(), None]


def block_args(**kw):
    a = dict(x=far(0), z=far(1), wp=far(2), gate=far(3), w=far(4), x2=far(5), h=far(6), dtype=0, rows=10, D=64, eps=1e-6, rho=1.0)
    a.update(kw)
    return [*a.values(), None]


@pytest.mark.parametrize("bad", [dict(rows=0), dict(d=24), dict(d=512), dict(eps=0.0), dict(ot=3), dict(dtype=3), dict(o=None),
                                 dict(gate=far(1) + 8), dict(out=far(0)), dict(out=far(2)), dict(out=far(1) + 16)])
def test_gated_norm_refuses(L, bad):
    assert L.gdn_gated_norm(*gated_args(**bad)) == gdnspec.ERR_ARG


@pytest.mark.parametrize("bad", [dict(rows=0), dict(D=12), dict(D=8200), dict(eps=-1.0), dict(dtype=3), dict(x=None), dict(w=None),
                                 dict(wp=None), dict(gate=None), dict(x2=None), dict(z=None), dict(h=far(5)), dict(h=far(4)),
                                 dict(x2=far(0) + 16)])
def test_block_norm_refuses(L, bad):
    assert L.gdn_block_norm(*block_args(**bad)) == gdnspec.ERR_ARG


def test_size_queries(L):
    n = ctypes.c_size_t(0)
    assert L.gdn_norm_workspace_bytes(10, 12, ctypes.byref(n)) == gdnspec.ERR_ARG
    assert L.gdn_norm_workspace_bytes(10, 64, None) == gdnspec.ERR_ARG
    assert L.gdn_norm_workspace_bytes(10, 64, ctypes.byref(n)) == 0 and n.value >= 10 * 64 * 4
    assert L.gdn_seq_workspace_bytes(1, 64, 8, 3, 64, 64, 0, ctypes.byref(n)) == gdnspec.ERR_ARG
    states = (1000 // 64 + 3) * 8 * 256 * 256 * 4
    assert gdnspec.gdn_seq_record_bytes(3, 1000, 8, 8, 256, 256, "bf16") >= states
    assert gdnspec.gdn_seq_record_bytes(3, 1000, 8, 8, 256, 256, "f32") >= states
    assert gdnspec.gdn_seq_workspace_bytes(3, 0, 8, 8, 256, 256, "f32") >= 0
    assert gdnspec.strerror(gdnspec.ERR_INDEX) != "unknown status"


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    x = torch.zeros(4, 2, 16)
    g = torch.zeros(4, 2)
    with pytest.raises(ValueError):
        gdnspec.gdn_seq_forward(x, x, x, g, g, None, x, None, torch.zeros(1 << 20, dtype=torch.uint8))
    with pytest.raises(ValueError):
        gdnspec.gdn_seq_forward(x, x[:, :1], x, g, g, None, x, None, None)
    with pytest.raises(ValueError):
        gdnspec.gdn_seq_step(x, x, x, g, g[:1], torch.zeros(4, 2, 16, 16), x)
    with pytest.raises(ValueError):
        gdnspec.gdn_gated_norm(x, x, torch.zeros(8), x)
    with pytest.raises(ValueError):
        gdnspec.gdn_block_norm(x, None, None, None, torch.zeros(16), None, x[:2])
