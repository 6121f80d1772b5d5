"""Host-side logic of the step and q/k entry points, without a GPU: what is refused before any launch, byte
queries, and the rotation's frequencies against their definitions."""
import math

import numpy as np
import pytest

import linear_attention_gdn_gb300 as gdn

P = 4096   # an aligned address that is never read: every call here is refused, or has nothing to do


def refused(code, f, *a, **kw):
    with pytest.raises(gdn.GDNError) as e:
        f(*a, stream=0, **kw)
    assert e.value.status == code


def step(prob, q=P, k=P, v=P, g=P, beta=P, states=P, o=P, err=P, cu=P, slot_in=P, slot_out=P, f=gdn.gdn_step):
    return (f, prob, q, k, v, g, beta, states, o, err), dict(cu_seqlens_dev=cu, slot_in=slot_in, slot_out=slot_out)


@pytest.mark.parametrize("f", [gdn.gdn_step, gdn.gdn_kda_step])
@pytest.mark.parametrize("prob,change,code", [
    (dict(T=-1), {}, 1), (dict(N=-1), {}, 1), (dict(H=0), {}, 1), (dict(HV=0), {}, 1), (dict(slots=-1), {}, 1),
    (dict(H=2, HV=3), {}, 2), (dict(dk=64), {}, 2), (dict(dv=64), {}, 2), (dict(T=2 ** 31), {}, 2),
    (dict(dtype=3), {}, 1), (dict(dtype=-1), {}, 1),
    (dict(strides=(4, 0, 0)), {}, 1),          # rows overlap
    (dict(strides=(0, 132, 0)), {}, 1),        # not whole 16 bytes
    (dict(strides=(0, 0, -256)), {}, 1),
    ({}, dict(cu=None), 1),                    # five tokens of four sequences need their starts
    (dict(slots=3), dict(slot_in=None), 1),    # sequence n in slot n needs N slots
    ({}, dict(q=None), 1), ({}, dict(k=P + 8), 1), ({}, dict(v=None), 1), ({}, dict(g=None), 1), ({}, dict(beta=P + 4), 1),
    ({}, dict(states=None), 1), ({}, dict(o=None), 1), ({}, dict(err=None), 1),
])
def test_step_refusals(f, prob, change, code):
    p = gdn.step_problem(**{**dict(T=5, N=4, H=1, HV=2, slots=4), **prob})
    a, kw = step(p, f=f, **change)
    refused(code, *a, **kw)


def test_step_with_nothing_to_do():
    for p in (gdn.step_problem(0, 0, 1, 1, 0), gdn.step_problem(0, 3, 1, 1, 3)):
        gdn.gdn_step(p, *[None] * 7, P, cu_seqlens_dev=P, stream=0)


@pytest.mark.parametrize("prob,change,code", [
    (dict(T=-1), {}, 1), (dict(N=-1), {}, 1), (dict(C=0), {}, 1), (dict(C=12), {}, 1), (dict(W=0), {}, 1),
    (dict(W=5), {}, 2), (dict(slots=-1), {}, 1), (dict(dtype=7), {}, 1), (dict(T=2 ** 31), {}, 2),
    (dict(strides=(8, 0)), {}, 1), (dict(strides=(0, 20)), {}, 1),
    ({}, dict(cu=None), 1), (dict(slots=3), dict(slot_in=None), 1),
    ({}, dict(x=None), 1), ({}, dict(w=None), 1), ({}, dict(b=P + 4), 1), ({}, dict(window=None), 1), ({}, dict(y=P + 2), 1),
    ({}, dict(err=None), 1),
])
def test_conv_step_refusals(prob, change, code):
    p = gdn.conv_step_problem(**{**dict(T=5, N=4, C=16, slots=4), **prob})
    a = {**dict(x=P, w=P, b=P, window=P, y=P, err=P, cu=P, slot_in=P), **change}
    refused(code, gdn.gdn_conv1d_step, p, a["x"], a["w"], a["b"], a["window"], a["y"], a["err"], cu_seqlens_dev=a["cu"],
            slot_in=a["slot_in"])


QK = dict(T=5, HQ=2, HK=1, D=128)


@pytest.mark.parametrize("prob,code", [
    (dict(T=-1), 1), (dict(HQ=-1), 1), (dict(HK=-1), 1), (dict(D=0), 1), (dict(rot=3), 1), (dict(rot=130), 1),
    (dict(rot=-2), 1), (dict(layout=2), 1), (dict(norm=3), 1), (dict(dtype=3), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(D=514), 2), (dict(T=2 ** 31), 2), (dict(HQ=65536), 2),
])
def test_qk_bad_problems(prob, code):
    p = gdn.qk_problem(**{**QK, **prob})
    with pytest.raises(gdn.GDNError) as e:
        gdn.gdn_qk_workspace_bytes(p)
    assert e.value.status == code
    refused(code, gdn.gdn_qk_norm_rope_fwd, p, P, P, P, P, P, P, P, P, P)
    refused(code, gdn.gdn_qk_norm_rope_bwd, p, *[P] * 14, ws_bytes=1 << 30)


@pytest.mark.parametrize("prob,at,value", [
    ({}, 0, None), ({}, 1, None), ({}, 4, None), ({}, 4, P + 4), ({}, 7, None), ({}, 8, None), ({}, 0, P + 1),
    (dict(q_strides=(-128, 0)), 0, P), (dict(k_strides=(0, 64), HK=2), 0, P), (dict(qo_strides=(100, 128)), 0, P),
])
def test_qk_bad_arguments(prob, at, value):
    p = gdn.qk_problem(**{**QK, **prob})
    a = [P] * 9
    a[at] = value
    refused(1, gdn.gdn_qk_norm_rope_fwd, p, *a)
    b = [P] * 14
    b[at] = value
    refused(1, gdn.gdn_qk_norm_rope_bwd, p, *b, ws_bytes=1 << 30)


def test_qk_documents_and_workspace():
    refused(1, gdn.gdn_qk_norm_rope_fwd, gdn.qk_problem(**QK), P, P, P, P, P, None, P, P, P)   # cu_seqlens of no documents
    p = gdn.qk_problem(**QK)
    need = gdn.gdn_qk_workspace_bytes(p)
    assert need > 0 and need % (2 * 128 * 4) == 0
    refused(3, gdn.gdn_qk_norm_rope_bwd, p, *[P] * 14, ws_bytes=need - 1)
    refused(1, gdn.gdn_qk_norm_rope_bwd, p, *[P] * 13, None, ws_bytes=need)
    refused(1, gdn.gdn_qk_norm_rope_bwd, p, *[P] * 11, P + 2, P, P, ws_bytes=need)


def test_frequencies():
    rot = 64
    plain = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    f, m = gdn.gdn_rope_frequencies(rot)
    assert np.allclose(f, plain, rtol=1e-14) and m == 1.0
    f, m = gdn.gdn_rope_frequencies(rot, scaling=gdn.ROPE_LINEAR, factor=4.0)
    assert np.allclose(f, plain / 4, rtol=1e-14) and m == 1.0
    f, _ = gdn.gdn_rope_frequencies(rot, scaling=gdn.ROPE_BASE, factor=8.0)
    assert f[0] == 1.0 and math.isclose(f[-1], plain[-1] / 8, rel_tol=1e-12)
    f, m = gdn.gdn_rope_frequencies(rot, scaling=gdn.ROPE_PARTS, factor=8.0, original=4096)
    turns = plain * 4096 / (2 * np.pi)
    # whole pairs outside the ramp, whose ends are rounded outwards to pair indexes
    assert np.allclose(f[turns > 32 * 2], plain[turns > 32 * 2], rtol=1e-14)
    assert np.allclose(f[turns < 0.5], plain[turns < 0.5] / 8, rtol=1e-14)
    assert (f <= plain * (1 + 1e-14)).all() and (f >= plain / 8 * (1 - 1e-14)).all() and (np.diff(f) < 0).all()
    assert math.isclose(m, 0.1 * math.log(8.0) + 1, rel_tol=1e-6)
    assert len(gdn.gdn_rope_frequencies(0)[0]) == 0


@pytest.mark.parametrize("a", [dict(rot=3), dict(rot=-2), dict(rot=8, base=0.0), dict(rot=8, base=float("inf")),
                               dict(rot=8, scaling=4), dict(rot=8, scaling=1, factor=0.0),
                               dict(rot=8, scaling=1, factor=float("nan")), dict(rot=2, scaling=2, factor=2.0),
                               dict(rot=8, scaling=3, factor=0.5), dict(rot=8, scaling=3, factor=2.0, original=0.0),
                               dict(rot=8, scaling=3, factor=2.0, fast=0.5, slow=1.0)])
def test_bad_frequencies(a):
    with pytest.raises(gdn.GDNError) as e:
        gdn.gdn_rope_frequencies(**a)
    assert e.value.status == 1
