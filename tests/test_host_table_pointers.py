"""Tables, counters and weights that do not lie on their element's boundary are refused before any launch: a kernel's load
from there would be a misaligned address."""
import pytest

import linear_attention_gdn_gb300 as gdn
from tests.test_host_step_qk import P, QK, refused


@pytest.mark.parametrize("off", [1, 2])
@pytest.mark.parametrize("name", ["cu_seqlens_dev", "slot_in", "slot_out", "err"])
@pytest.mark.parametrize("f", [gdn.gdn_step, gdn.gdn_kda_step, gdn.gdn_conv1d_step])
def test_step_tables(f, name, off):
    tables = dict(cu_seqlens_dev=P, slot_in=P, slot_out=P)
    err = P + off if name == "err" else P
    if name != "err":
        tables[name] = P + off
    if f is gdn.gdn_conv1d_step:
        refused(1, f, gdn.conv_step_problem(5, 4, 16, 4), P, P, P, P, P, err, **tables)
    else:
        refused(1, f, gdn.step_problem(5, 4, 1, 2, 4), *[P] * 7, err, **tables)


@pytest.mark.parametrize("off", [1, 2])
@pytest.mark.parametrize("at", [2, 3, 5, 6])   # wq, wk, positions, cu_seqlens_dev
def test_qk_weights_and_tables(at, off):
    p = gdn.qk_problem(**QK, N=1)
    a = [P] * 14
    a[at] += off
    refused(1, gdn.gdn_qk_norm_rope_fwd, p, *a[:9])
    refused(1, gdn.gdn_qk_norm_rope_bwd, p, *a, ws_bytes=1 << 30)


def test_tables_of_whole_words_are_taken():
    """Tables need no more than that (a view from the second entry on): a call with nothing to do takes them."""
    gdn.gdn_step(gdn.step_problem(0, 3, 1, 1, 3), *[P] * 7, P + 4, cu_seqlens_dev=P + 4, slot_in=P + 8, slot_out=P + 12,
                 stream=0)
    gdn.gdn_conv1d_step(gdn.conv_step_problem(0, 3, 16, 3), *[P] * 5, P + 4, cu_seqlens_dev=P + 4, slot_in=P + 8,
                        slot_out=P + 12, stream=0)
    gdn.gdn_qk_norm_rope_fwd(gdn.qk_problem(**{**QK, "T": 0}), P, P, P + 4, P + 4, P, P + 4, P + 4, P, P, stream=0)
