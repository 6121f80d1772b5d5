"""Host-side logic of the linear attention, the residual stream's norm and the step's tables, without a GPU: what is
refused before any launch, and byte queries."""
import numpy as np
import pytest

import linear_attention_gdn_gb300 as gdn
from tests.test_host_step_qk import P, refused, step

CU = np.array([0, 3, 5], np.int32)
LA = dict(T=5, N=2, H=1, HV=2)


def fwd(prob, cu=CU, ws_bytes=1 << 30, **change):
    a = {**dict(q=P, k=P, v=P, decay=P, cu_dev=P, s_in=P, o=P, s_out=P, err=P, ws=P), **change}
    return (gdn.gdn_la_fwd, prob, a["q"], a["k"], a["v"], a["decay"], a["cu_dev"], cu, a["s_in"], a["o"], a["s_out"], a["err"],
            a["ws"], ws_bytes)


def bwd(prob, cu=CU, ws_bytes=1 << 30, **change):
    a = {**dict(q=P, k=P, v=P, decay=P, cu_dev=P, s_in=P, dO=P, ds_out=P, dq=P, dk=P, dv=P, ds_in=P, err=P, ws=P), **change}
    return (gdn.gdn_la_bwd, prob, a["q"], a["k"], a["v"], a["decay"], a["cu_dev"], cu, a["s_in"], a["dO"], a["ds_out"], a["dq"],
            a["dk"], a["dv"], a["ds_in"], a["err"], a["ws"], ws_bytes)


@pytest.mark.parametrize("call", [fwd, bwd])
@pytest.mark.parametrize("prob,cu,code", [
    (dict(T=-1), CU, 1), (dict(N=0), [0], 1), (dict(H=0), CU, 1), (dict(HV=0), CU, 1), (dict(segment=-1), CU, 1),
    (dict(H=2, HV=3), CU, 2), (dict(dk=64), CU, 2), (dict(dv=256), CU, 2), (dict(T=2 ** 30, N=1), [0, 2 ** 30], 2),
    ({}, [0, 3, 4], 1), ({}, [1, 3, 5], 1), ({}, [0, 6, 5], 1),
    (dict(strides=(64, 0, 0)), CU, 1), (dict(strides=(0, 132, 0)), CU, 1), (dict(strides=(0, 0, -256)), CU, 1),
])
def test_la_bad_problems(call, prob, cu, code):
    p = gdn.la_problem(**{**LA, **prob})
    refused(code, *call(p, cu=np.array(cu, np.int32)))
    if "strides" not in prob:
        with pytest.raises(gdn.GDNError) as e:
            gdn.gdn_la_workspace_bytes(p, cu)
        assert e.value.status == code


@pytest.mark.parametrize("call,change", [
    (c, {n: v}) for c, names in ((fwd, ("q", "k", "v", "o")), (bwd, ("q", "k", "v", "dO", "dq", "dk", "dv")))
    for n in names for v in (None, P + 8)] + [
    (c, x) for c in (fwd, bwd) for x in (dict(decay=None), dict(decay=P + 2), dict(cu_dev=None), dict(cu_dev=P + 1),
                                         dict(err=None), dict(s_in=P + 4))] + [
    (fwd, dict(s_out=P + 8)), (bwd, dict(ds_out=P + 4)), (bwd, dict(ds_in=P + 8))])
def test_la_bad_arguments(call, change):
    refused(1, *call(gdn.la_problem(**LA), **change))


def test_la_workspace():
    one = gdn.la_problem(**LA)
    # FP32 sums of dq and dk over the value heads of a group: a tile to a chunk, the counts of heads that are in them, a ticket
    for H, HV in ((1, 2), (2, 2), (1, 8), (2, 32), (1, 11)):
        b = 0 if H == HV else 2 * ((0 + 2 + 1) * H * (65536 + 4) + 4)
        assert gdn.gdn_la_workspace_bytes(gdn.la_problem(5, 2, H, HV), CU) == (0, b)
    cu = [0, 300, 300, 301]
    cut = gdn.la_problem(301, 3, 2, 2, segment=2)                    # segments: 2, 1, 1
    f, b = gdn.gdn_la_workspace_bytes(cut, cu)
    assert (f, b) == (4 * 2 * 65536, 2 * 4 * 2 * 65536)
    refused(3, *fwd(cut, np.array(cu, np.int32), ws_bytes=f - 1))
    refused(3, *bwd(cut, np.array(cu, np.int32), ws_bytes=b - 1))
    refused(1, *fwd(cut, np.array(cu, np.int32), ws=P + 8))
    refused(1, *bwd(cut, np.array(cu, np.int32), ws=None))
    with pytest.raises(ValueError):
        gdn.gdn_la_fwd(one, *[P] * 5, CU[:2], P, P, P, P, P, 0, stream=0)


@pytest.mark.parametrize("cu", [[0, 5], [0], [], [[0, 3, 5]], 5])
def test_la_tables_too_short_for_the_documents(cu):
    """No entry point reads past the table that it is given."""
    p = gdn.la_problem(**LA)
    with pytest.raises(ValueError):
        gdn.gdn_la_workspace_bytes(p, cu)
    for call in (fwd, bwd):
        f, *a = call(p, cu=cu)
        with pytest.raises(ValueError):
            f(*a, stream=0)


def test_la_cuts_long_documents_only_where_heads_are_few():
    many = gdn.la_problem(8192 * 8, 8, 16, 48)
    assert gdn.gdn_la_workspace_bytes(many, np.arange(9) * 8192)[0] == 0
    few = gdn.la_problem(32768, 1, 4, 4)
    assert gdn.gdn_la_workspace_bytes(few, [0, 32768])[0] >= 8 * 4 * 65536


def test_la_with_nothing_to_do():
    gdn.gdn_la_fwd(gdn.la_problem(0, 1, 1, 1), None, None, None, P, P, np.zeros(2, np.int32), P, None, None, P, None, 0, stream=0)
    gdn.gdn_la_bwd(gdn.la_problem(0, 1, 1, 1), None, None, None, P, P, np.zeros(2, np.int32), P, None, P, None, None, None, None,
                   P, None, 0, stream=0)


@pytest.mark.parametrize("prob,change,code", [
    (dict(l2norm=True), {}, 2), (dict(T=-1), {}, 1), (dict(H=2, HV=3), {}, 2), (dict(dk=64), {}, 2), (dict(dtype=3), {}, 1),
    (dict(strides=(4, 0, 0)), {}, 1), ({}, dict(cu=None), 1), (dict(slots=3), dict(slot_in=None), 1),
    ({}, dict(q=None), 1), ({}, dict(k=P + 8), 1), ({}, dict(v=None), 1), ({}, dict(g=None), 1), ({}, dict(g=P + 2), 1),
    ({}, dict(states=None), 1), ({}, dict(o=None), 1), ({}, dict(err=None), 1), ({}, dict(err=P + 2), 1),
])
def test_la_step_refusals(prob, change, code):
    p = gdn.step_problem(**{**dict(T=5, N=4, H=1, HV=2, slots=4, l2norm=False), **prob})
    a, kw = step(p, **change)
    _, p, q, k, v, g, beta, states, o, err = a
    refused(code, gdn.gdn_la_step, p, q, k, v, g, states, o, err, **kw)


@pytest.mark.parametrize("prob,code", [
    (dict(T=-1), 1), (dict(C=0), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(dtype=3), 1), (dict(group=-32), 1),
    (dict(C=100, group=32), 1), (dict(group=16), 2), (dict(C=512, group=256), 2), (dict(T=2 ** 31), 2), (dict(C=2 ** 21), 2),
])
def test_norm_bad_problems(prob, code):
    p = gdn.norm_problem(**{**dict(T=4, C=64), **prob})
    refused(code, gdn.gdn_add_norm_fwd, p, P, P, P, P, P, P, P)
    refused(code, gdn.gdn_add_norm_bwd, p, P, P, P, P, P, P, P, 1 << 30)
    with pytest.raises(gdn.GDNError):
        gdn.gdn_add_norm_workspace_bytes(p)


@pytest.mark.parametrize("change", [
    dict(x=None), dict(x=P + 1), dict(r=P + 1), dict(h=None), dict(h=P + 1), dict(y=P + 1), dict(w=None), dict(w=P + 2),
    dict(y8=None), dict(scales=None), dict(scales=P + 2), dict(r=None, h=None, y=None, y8=None, scales=None)])
def test_norm_bad_arguments(change):
    a = {**dict(x=P, r=P, w=P, h=P, y=P, y8=P, scales=P), **change}
    refused(1, gdn.gdn_add_norm_fwd, gdn.norm_problem(4, 64), *a.values())


@pytest.mark.parametrize("prob", [dict(strides=(63, 0, 0, 0)), dict(strides=(0, 0, 0, -64)), dict(strides=(0, 1, 0, 0))])
def test_norm_bad_strides(prob):
    p = gdn.norm_problem(4, 64, **prob)
    refused(1, gdn.gdn_add_norm_fwd, p, *[P] * 7)
    refused(1, gdn.gdn_add_norm_bwd, p, *[P] * 7, 1 << 30)


@pytest.mark.parametrize("change,code", [
    (dict(h=None), 1), (dict(w=None), 1), (dict(dy=P + 1), 1), (dict(dres=P + 1), 1), (dict(dx=None), 1), (dict(dw=P + 2), 1),
    (dict(ws=None), 1), (dict(bytes=0), 3)])
def test_norm_backward_bad_arguments(change, code):
    a = {**dict(h=P, w=P, dy=P, dres=P, dx=P, dw=P, ws=P, bytes=1 << 30), **change}
    refused(code, gdn.gdn_add_norm_bwd, gdn.norm_problem(4, 64), *a.values())


TABLES = dict(N=3, T=8, block=4, max_blocks=5, slots=9)


@pytest.mark.parametrize("prob,code", [
    (dict(N=-1), 1), (dict(T=-1), 1), (dict(block=0), 1), (dict(max_blocks=-1), 1), (dict(slots=-1), 1),
    (dict(N=16385), 2), (dict(block=1 << 20, max_blocks=1 << 11), 2), (dict(T=2 ** 31 - 1), 2),
])
def test_tables_bad_problems(prob, code):
    refused(code, gdn.gdn_step_tables, gdn.tables_problem(**{**TABLES, **prob}), *[P] * 12)


@pytest.mark.parametrize("at,value", [(i, None) for i in range(12) if i != 8] + [(i, P + 2) for i in range(12)])
def test_tables_bad_arguments(at, value):
    a = [P] * 12
    a[at] = value
    refused(1, gdn.gdn_step_tables, gdn.tables_problem(**TABLES), *a)
